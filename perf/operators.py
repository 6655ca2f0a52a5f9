"""The operators of unbounded streaming sessions, as cases that can be run and timed: attention with a
sliding window and sinks over a paged KV cache (prompts and single frames), and the cache's page calls
(resize, fork, compact).

A case names sizes only; `prepare` makes the tensors, `run` makes one pass.  With `own` false a pass is the
operator's plain form in elementary torch operations; with `own` true it is the package's call.

Layouts: k and v [layers][pages][kv_heads][page][head_dim], table int32 [seqs][columns] (the page of
positions column * page ..., -1: none), lens int32 [seqs], refs int32 [pages] (how many table entries name
the page).  A query at position p sees the keys t <= p with t < sinks or t > p - window (window 0: all).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    nano = dict(q_heads=40, kv_heads=8, head_dim=128, page=64, dtype="bf16")
    mid = dict(q_heads=32, kv_heads=8, head_dim=64)
    return [
        # one caller's 80 ms frame: the call whose latency the caller waits for
        dict(name="frame, 1 session", op="attend", sessions=1, rows_lo=1, rows_hi=1, ctx_lo=2000, ctx_hi=2000,
             window=1024, sinks=4, spread=1, **nano),
        # a frame of 16 ragged sessions, the batch the backbone serves
        dict(name="frame, 16 sessions", op="attend", sessions=16, rows_lo=1, rows_hi=1, ctx_lo=500, ctx_hi=6000,
             window=4096, sinks=64, spread=2, **nano),
        # a frame of many sessions that keep their whole context (no window)
        dict(name="frame, 64 long sessions", op="attend", sessions=64, rows_lo=1, rows_hi=1, ctx_lo=1, ctx_hi=32000,
             window=0, sinks=0, spread=3, page=128, dtype="fp16", **mid),
        # a short opening context of odd length through the smallest stack's heads
        dict(name="prompt, 257 rows", op="attend", sessions=1, rows_lo=257, rows_hi=257, ctx_lo=0, ctx_hi=0,
             window=100, sinks=3, spread=4, q_heads=8, kv_heads=2, head_dim=32, page=16, dtype="fp16"),
        # an opening context of twice the usual length
        dict(name="prompt, 8192 rows", op="attend", sessions=1, rows_lo=8192, rows_hi=8192, ctx_lo=0, ctx_hi=0,
             window=4096, sinks=64, spread=5, **nano),
        # sessions that hand in blocks of very different lengths behind what they hold
        dict(name="prompt, 12 ragged blocks", op="attend", sessions=12, rows_lo=1, rows_hi=900, ctx_lo=0, ctx_hi=6000,
             window=2048, sinks=16, spread=6, page=32, dtype="bf16", **mid),
        # the bookkeeping of one frame: 16 sessions take one more position each
        dict(name="resize, 16 sessions", op="resize", sessions=16, mode="frame", ctx_lo=500, ctx_hi=6000, window=4096,
             sinks=64, spread=7, shared=0, layers=1, pages=4096, columns=512, kv_heads=2, head_dim=32, page=64,
             dtype="bf16"),
        # a server's turn: of 512 sessions some end, some take a block, some one frame; some write behind a
        # shared page and get a copy of it
        dict(name="resize, 512 sessions", op="resize", sessions=512, mode="turn", ctx_lo=1, ctx_hi=6000, window=2048,
             sinks=16, spread=8, shared=16, layers=4, pages=65536, columns=1024, kv_heads=2, head_dim=32, page=32,
             dtype="bf16"),
        # one opening context handed to 15 sessions
        dict(name="fork, 1 to 15", op="fork", sessions=16, sources=1, ctx_lo=1000, ctx_hi=1000, window=0, sinks=0,
             spread=9, layers=4, pages=512, columns=64, kv_heads=8, head_dim=128, page=64, dtype="bf16", ssm_layers=0,
             ssm_heads=128, ssm_dim=80, ssm_state=128),
        # eight sessions of the hybrid copied: pages and the Mamba-2 states
        dict(name="fork, 8 with states", op="fork", sessions=16, sources=8, ctx_lo=500, ctx_hi=6000, window=4096,
             sinks=64, spread=10, layers=4, pages=2048, columns=128, kv_heads=8, head_dim=128, page=64, dtype="bf16",
             ssm_layers=27, ssm_heads=128, ssm_dim=80, ssm_state=128),
        # a small pool drawn together
        dict(name="compact, 256 pages", op="compact", sessions=12, ctx_lo=1, ctx_hi=500, spread=11, layers=1, pages=256,
             columns=32, kv_heads=2, head_dim=32, page=16, dtype="fp16"),
        # a pool of some GB drawn together before part of it is given back
        dict(name="compact, 4096 pages", op="compact", sessions=48, ctx_lo=500, ctx_hi=6000, spread=12, layers=4,
             pages=4096, columns=128, kv_heads=8, head_dim=128, page=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "resize", "fork", "compact"])
    heads = rng.choice([(40, 8, 128), (32, 8, 64), (8, 2, 32), (16, 4, 64), (32, 4, 128), (5, 1, 128), (8, 4, 256),
                        (12, 12, 64)])
    c = dict(op=op, q_heads=heads[0], kv_heads=heads[1], head_dim=heads[2], page=rng.choice([16, 32, 64, 128]),
             dtype=rng.choice(["bf16", "fp16"]), spread=rng.randrange(1 << 20),
             window=rng.choice([0, _log(rng, 1, 6000), _log(rng, 100, 6000)]), sinks=rng.choice([0, _log(rng, 1, 200)]))
    if op == "attend" and rng.random() < 0.5:
        n = _log(rng, 1, 64)
        c.update(sessions=n, rows_lo=1, rows_hi=1, ctx_lo=1, ctx_hi=_log(rng, 100, min(30000, 700000 // n)))
    elif op == "attend":
        n = _log(rng, 1, 16)
        c.update(sessions=n, rows_lo=1, rows_hi=_log(rng, 2, 6000 // n), ctx_lo=0, ctx_hi=_log(rng, 1, 16000 // n))
    else:
        del c["q_heads"]
        c.update(layers=rng.randint(1, 4), columns=1024, kv_heads=rng.choice([1, 2, 4, 8]), head_dim=rng.choice([32, 64, 128]))
        if op == "resize":
            c.update(sessions=_log(rng, 1, 300), mode=rng.choice(["frame", "turn"]), ctx_lo=1, ctx_hi=_log(rng, 100, 6000),
                     shared=rng.choice([0, 1, 4]), layers=1, kv_heads=2, head_dim=32)
            c["pages"] = c["sessions"] * ((c["ctx_hi"] + 4096) // c["page"] + 4)
        elif op == "fork":
            n = rng.randint(2, 24)
            c.update(sessions=n, sources=rng.randint(1, n // 2), ctx_lo=1, ctx_hi=_log(rng, 30, 6000), ssm_layers=rng.choice([0, 1, 6]),
                     ssm_heads=8, ssm_dim=rng.choice([16, 80]), ssm_state=rng.choice([16, 128]))
            c["pages"] = n * (c["ctx_hi"] // c["page"] + 2)
        else:
            del c["window"], c["sinks"]
            c.update(sessions=rng.randint(1, 40), ctx_lo=1, ctx_hi=_log(rng, 30, 3000))
            c["pages"] = int((c["sessions"] * (c["ctx_hi"] // c["page"] + 1) + 4) * rng.uniform(1.0, 3.0))
    return c


# ---- what a case's sizes say: lengths by session, the same for every seed ---------------------------


def _spread(c, lo, hi, n, salt):
    r = random.Random(c["spread"] * 4 + salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _targets(c, lens):
    if c["mode"] == "frame":
        return [n + 1 for n in lens]
    r = random.Random(c["spread"] * 4 + 3)
    kinds = [r.choice(["end", "block", "frame", "frame", "back"]) for _ in lens]
    top = c["columns"] * c["page"]
    return [{"end": 0, "block": min(top, n + r.randint(1, 4096)), "frame": min(top, n + 1), "back": r.randint(0, n)}[k]
            for k, n in zip(kinds, lens)]


def _columns_kept(c, n, page):
    """the columns of a session of n positions that hold a page: the sinks' and the window's"""
    have = -(-n // page)
    if not c.get("window"):
        return list(range(have))
    first = -(-c["sinks"] // page)
    return [k for k in range(have) if k < first or (k + 1) * page - 1 > n - 1 - c["window"]]


def _cache(c, lens, g, pages, columns, layers):
    """A pool whose pages are named by the tables in random order.  The ints live in one tensor, so that a pass
    that changes them can put them back in one copy."""
    page, n_seqs = c["page"], len(lens)
    shape = (layers, pages, c["kv_heads"], page, c["head_dim"])
    dt = DTYPES[c["dtype"]]
    k = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    v = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    rows, cols = [], []
    for s, n in enumerate(lens):
        kept = _columns_kept(c, n, page)
        rows += [s] * len(kept)
        cols += kept
    order = torch.randperm(pages, generator=g, device="cuda")[: len(rows)].int()
    up = lambda n: -(-n // 4) * 4  # noqa: E731  (16-byte aligned views)
    ints = torch.zeros(up(n_seqs * columns) + up(n_seqs) + pages, dtype=torch.int32, device="cuda")
    a, b = up(n_seqs * columns), up(n_seqs * columns) + up(n_seqs)
    table, seq_len, refs = ints[: n_seqs * columns].view(n_seqs, columns), ints[a: a + n_seqs], ints[b:]
    table.fill_(-1)
    if rows:
        table[torch.tensor(rows, device="cuda"), torch.tensor(cols, device="cuda")] = order
        refs[order.long()] = 1
    seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    return dict(k=k, v=v, ints=ints, table=table, lens=seq_len, refs=refs, page=page, window=c.get("window", 0),
                sinks=c.get("sinks", 0))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"op": c["op"]}
    if c["op"] == "attend":
        rows = _spread(c, c["rows_lo"], c["rows_hi"], c["sessions"], 0)
        ctx = _spread(c, c["ctx_lo"], c["ctx_hi"], c["sessions"], 1)
        lens = [a + b for a, b in zip(ctx, rows)]
        columns = -(-max(lens) // c["page"]) + 1
        # the first new row sees from ctx - window on: pages are kept for a window that reaches there from the end
        s.update(_cache(dict(c, window=c["window"] and c["window"] + max(rows)), lens, g,
                        sum(-(-n // c["page"]) for n in lens) + 3, columns, 1))
        s["window"] = c["window"]
        total, dt = sum(rows), DTYPES[c["dtype"]]
        hq, hk, d = c["q_heads"], c["kv_heads"], c["head_dim"]
        # the rows as a projection leaves them: q, k and v of a row behind one another
        qkv = torch.empty((total, (hq + 2 * hk) * d), dtype=dt, device="cuda").normal_(generator=g)
        s["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
        s["k_new"] = qkv[:, hq * d: (hq + hk) * d].unflatten(1, (hk, d))
        s["v_new"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        s["out"] = torch.zeros((total, hq, d), dtype=dt, device="cuda")
        s["pos"] = _ints(ctx)
        starts = [0]
        for r in rows:
            starts.append(starts[-1] + r)
        s["cu_rows"] = None if c["rows_hi"] == 1 else _ints(starts)
        s["most"] = max(rows)
        q_heads = hq
    elif c["op"] == "resize":
        lens = _spread(c, c["ctx_lo"], c["ctx_hi"], c["sessions"], 1)
        s.update(_cache(c, lens, g, c["pages"], c["columns"], c["layers"]))
        for i in range(min(c["shared"], c["sessions"] // 2)):  # the second of a pair holds the first's pages
            a, b = 2 * i, 2 * i + 1
            old = s["table"][b]
            s["refs"].scatter_(0, old.clamp(min=0).long()[old >= 0], 0)
            s["table"][b] = s["table"][a]
            s["lens"][b] = s["lens"][a]
            held = s["table"][a]
            s["refs"].scatter_(0, held.long()[held >= 0], 2)
            lens[b] = lens[a]
        s["to"] = _ints(_targets(c, lens))
        s["pos"] = torch.zeros(c["sessions"], dtype=torch.int32, device="cuda")
    elif c["op"] == "fork":
        n, m = c["sessions"], c["sources"]
        lens = _spread(c, c["ctx_lo"], c["ctx_hi"], m, 1) + [0] * (n - m)
        s.update(_cache(c, lens, g, c["pages"], c["columns"], c["layers"]))
        s["dst"] = _ints(list(range(m, n)))
        s["src"] = _ints([i % m for i in range(n - m)])
        s["done"] = torch.zeros(n - m, dtype=torch.int32, device="cuda")
        s["states"] = None
        if c["ssm_layers"]:
            s["states"] = torch.empty((c["ssm_layers"], n, c["ssm_heads"], c["ssm_dim"], c["ssm_state"]), device="cuda").normal_(generator=g)
    else:
        lens = _spread(c, c["ctx_lo"], c["ctx_hi"], c["sessions"], 1)
        s.update(_cache(c, lens, g, c["pages"], c["columns"], c["layers"]))
        s["live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if c["op"] != "attend":
        s["ints_before"] = s["ints"].clone()
        q_heads = c["kv_heads"]
    if own:
        import attention_frame_decode_b200 as vc
        s["cache"] = vc.PagedCache(s["k"], s["v"], s["table"], s["lens"], s["refs"], q_heads=q_heads, window=s["window"],
                                   sinks=s["sinks"])
        if c["op"] == "fork":
            s["parts"] = vc.session_parts([s["states"]]) if s["states"] is not None else None
    return s


# ---- the plain forms ---------------------------------------------------------------------------


def _plain_attend(s):
    q, table, page, window, sinks = s["q"], s["table"].long(), s["page"], s["window"], s["sinks"]
    k_pool, v_pool = s["k"][0], s["v"][0]
    total, hq, d = q.shape
    n, hk = table.shape[0], k_pool.shape[1]
    dev = q.device
    row = torch.arange(total, device=dev)
    starts = torch.arange(n + 1, device=dev) if s["cu_rows"] is None else s["cu_rows"].long()
    session = torch.searchsorted(starts, row, right=True) - 1
    nth = row - starts[session]
    at = s["pos"].long()[session] + nth
    # the new keys and values into their pages
    to = table[session, at // page]
    k_pool[to, :, at % page] = s["k_new"]
    v_pool[to, :, at % page] = s["v_new"]
    # every session's positions in order, in 32 bits
    length = table.shape[1] * page
    t = torch.arange(length, device=dev)
    held = (table.clamp(min=0)[:, t // page] >= 0) & (table[:, t // page] >= 0) & (t < (s["pos"].long() + starts[1:] - starts[:-1])[:, None])
    keys = k_pool[table.clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(n, hk, length, d).float()
    values = v_pool[table.clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(n, hk, length, d).float()
    values.mul_(held[:, None, :, None])
    # the rows of a session side by side, padded to the longest
    padded = torch.zeros((n, s["most"], hq, d), device=dev)
    padded[session, nth] = q.float()
    x = padded.reshape(n, s["most"], hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    scores = (x @ keys.transpose(-1, -2)).mul_(d ** -0.5).view(n, hk, hq // hk, s["most"], length)
    p = (s["pos"].long()[:, None] + torch.arange(s["most"], device=dev))[:, :, None]
    seen = held[:, None] & (t <= p)
    if window:
        seen &= (t < sinks) | (t > p - window)
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    weights = scores.sub_(top).exp_()
    total_weight = weights.sum(-1, keepdim=True)
    out = (weights.view(n, hk, -1, length) @ values).view(n, hk, hq // hk, s["most"], d) / total_weight.clamp(min=1e-30)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, s["most"], hq, d)
    s["out"].copy_(out[session, nth])
    return {"out": s["out"], "k": s["k"], "v": s["v"]}


def _copy_rows(s, src, dst, count):
    """the first count rows (of every head and layer) of the pages src into dst"""
    keep = (torch.arange(s["page"], device=src.device) < count[:, None])[None, :, None, :, None]
    s["k"][:, dst] = torch.where(keep, s["k"][:, src], s["k"][:, dst])
    s["v"][:, dst] = torch.where(keep, s["v"][:, src], s["v"][:, dst])


def _add_refs(refs, pages, amount):
    """refs[pages] += amount where amount is not 0 (pages may repeat)"""
    refs.scatter_add_(0, pages.clamp(min=0).long().reshape(-1), amount.int().reshape(-1))


def _plain_resize(s):
    s["ints"].copy_(s["ints_before"])
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    to, have = s["to"].long(), lens.long()
    col = torch.arange(table.shape[1], device=to.device)
    start = torch.minimum(to, have)
    # a length inside a page that the window has given up is refused
    there = table.gather(1, (start // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0] >= 0
    good = there | (start % page == 0)
    to = torch.where(good, to, have)
    up = lambda x: (x + page - 1) // page  # noqa: E731
    drop = (col >= up(to)[:, None]) & (col < up(have)[:, None])
    if s["window"]:
        drop |= (col >= up(s["sinks"])) & ((col + 1) * page - 1 <= (start - s["window"])[:, None])
    drop &= (table >= 0) & good[:, None]
    _add_refs(refs, table, -drop.int())
    table.masked_fill_(drop, -1)
    grow = (to > have) & (to <= table.shape[1] * page)
    last = (have // page).clamp(max=table.shape[1] - 1)
    last_page = table.gather(1, last[:, None])[:, 0].long()
    shared = grow & (have % page != 0) & (last_page >= 0) & (refs[last_page.clamp(min=0)] > 1)
    want = (col >= up(have)[:, None]) & (col < up(to)[:, None]) & grow[:, None]
    want |= shared[:, None] & (col == last[:, None])
    need = want.sum(1)
    free = torch.nonzero(refs == 0)[:, 0]
    fits = (to <= table.shape[1] * page) & ((need == 0) | (need.cumsum(0) <= free.numel()))
    want &= fits[:, None]
    table[want] = free[: int(want.sum())].int()
    refs.scatter_add_(0, free, (torch.arange(free.numel(), device=to.device) < want.sum()).int())
    shared &= fits
    _add_refs(refs, last_page, -shared.int())
    _copy_rows(s, last_page[shared], table.gather(1, last[:, None])[:, 0].long()[shared], (have % page)[shared])
    s["pos"].copy_(torch.where(fits & good, start, -1))
    lens.copy_(torch.where(fits, to, have))
    return {"k": s["k"], "v": s["v"], "ints": s["ints"], "pos": s["pos"]}


def _plain_fork(s):
    s["ints"].copy_(s["ints_before"])
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    src, dst = s["src"].long(), s["dst"].long()
    _add_refs(refs, table[dst], -(table[dst] >= 0).int())
    table[dst] = -1
    have = lens[src].long()
    col = torch.arange(table.shape[1], device=src.device)
    theirs = table[src]
    whole = (col < (have // page)[:, None]) & (theirs >= 0)
    last = (have // page).clamp(max=table.shape[1] - 1)
    last_page = theirs.gather(1, last[:, None])[:, 0].long()
    part = (have % page != 0) & (last_page >= 0)
    free = torch.nonzero(refs == 0)[:, 0]
    fits = ~part | (part.cumsum(0) <= free.numel())
    part &= fits
    whole &= fits[:, None]
    mine = torch.where(whole, theirs, -1)
    new = free[(part.cumsum(0) - 1).clamp(min=0)].int()
    mine.scatter_(1, last[:, None], torch.where(part, new, mine.gather(1, last[:, None])[:, 0])[:, None])
    table[dst] = mine
    _add_refs(refs, theirs, whole.int())
    _add_refs(refs, new, part.int())
    _copy_rows(s, last_page[part], new[part].long(), (have % page)[part])
    lens[dst] = torch.where(fits, have, 0).int()
    s["done"].copy_(fits.int())
    got = {"k": s["k"], "v": s["v"], "ints": s["ints"], "done": s["done"]}
    if s["states"] is not None:
        s["states"][:, dst[fits]] = s["states"][:, src[fits]]
        got["states"] = s["states"]
    return got


def _plain_compact(s):
    s["ints"].copy_(s["ints_before"])
    table, refs = s["table"], s["refs"]
    live = refs > 0
    count = live.sum()
    page = torch.arange(refs.numel(), device=refs.device)
    source = torch.nonzero(live & (page >= count))[:, 0]
    hole = torch.nonzero(~live & (page < count))[:, 0]
    name = page.int()
    name[source] = hole.int()
    table.copy_(torch.where(table >= 0, name[table.clamp(min=0).long()], -1))
    refs[hole] = refs[source]
    refs[source] = 0
    s["k"][:, hole] = s["k"][:, source]
    s["v"][:, hole] = s["v"][:, source]
    s["live"][0] = count
    return {"k": s["k"], "v": s["v"], "ints": s["ints"], "live": s["live"]}


def run(state):
    s = state
    if not own:
        return {"attend": _plain_attend, "resize": _plain_resize, "fork": _plain_fork, "compact": _plain_compact}[s["op"]](s)
    cache = s["cache"]
    if s["op"] == "attend":
        cache.attend(0, s["q"], s["k_new"], s["v_new"], s["out"], s["pos"], cu_rows=s["cu_rows"])
        return {"out": s["out"], "k": s["k"], "v": s["v"]}
    s["ints"].copy_(s["ints_before"])
    if s["op"] == "resize":
        cache.resize(lens=s["to"], pos=s["pos"])
        return {"k": s["k"], "v": s["v"], "ints": s["ints"], "pos": s["pos"]}
    if s["op"] == "fork":
        cache.fork(s["src"], s["dst"], parts=s["parts"], done=s["done"])
        got = {"k": s["k"], "v": s["v"], "ints": s["ints"], "done": s["done"]}
        if s["states"] is not None:
            got["states"] = s["states"]
        return got
    cache.compact(live=s["live"])
    return {"k": s["k"], "v": s["v"], "ints": s["ints"], "live": s["live"]}


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    c = case
    d, hk = c["head_dim"], c["kv_heads"]
    row_bytes = 2 * 2 * hk * d  # one position's key and value in one layer
    if c["op"] == "attend":
        rows = _spread(c, c["rows_lo"], c["rows_hi"], c["sessions"], 0)
        ctx = _spread(c, c["ctx_lo"], c["ctx_hi"], c["sessions"], 1)
        w, sinks = c["window"] or 1 << 30, c["sinks"]
        pairs = old = 0
        for r, x in zip(rows, ctx):
            pairs += sum(min(p + 1, w) + max(0, min(sinks, p + 1 - w)) for p in range(x, x + r))
            old += min(x, w - 1) + max(0, min(sinks, x - (w - 1)))
        bytes_ = old * row_bytes + sum(rows) * (2 * row_bytes + 2 * 2 * c["q_heads"] * d)
        return {"bytes": bytes_, "flops": 4 * d * c["q_heads"] * pairs}
    page_bytes = row_bytes * c["page"] * c["layers"]
    if c["op"] == "resize":
        lens = _spread(c, c["ctx_lo"], c["ctx_hi"], c["sessions"], 1)
        to = _targets(c, lens)
        changed = sum(abs(-(-b // c["page"]) - -(-a // c["page"])) for a, b in zip(lens, to))
        # a length, a target and a position for each session; a table entry and a count, read and written, for each page
        return {"bytes": 16 * c["sessions"] + 16 * changed, "flops": 0}
    if c["op"] == "fork":
        lens = _spread(c, c["ctx_lo"], c["ctx_hi"], c["sources"], 1)
        have = [lens[i % c["sources"]] for i in range(c["sessions"] - c["sources"])]
        entries = sum(len(_columns_kept(c, n, c["page"])) for n in have)
        rows = sum(n % c["page"] for n in have)
        state = 4 * c["ssm_layers"] * c["ssm_heads"] * c["ssm_dim"] * c["ssm_state"]
        return {"bytes": 16 * entries + 2 * rows * row_bytes * c["layers"] + 2 * state * len(have) + 16 * len(have), "flops": 0}
    lens = _spread(c, c["ctx_lo"], c["ctx_hi"], c["sessions"], 1)
    live = sum(-(-n // c["page"]) for n in lens)
    moved = live * (c["pages"] - live) // c["pages"]  # of pages named in random order
    return {"bytes": 4 * c["pages"] + 4 * live + 12 * moved + 2 * moved * page_bytes, "flops": 0}


# ---- the definition in 64 bits ---------------------------------------------------------------------


def exact(case, seed):
    """Attention by its definition, session by session and head by head in 64 bits.  The page calls move and count,
    which whole numbers and equal bits settle: nothing is computed there."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    hk, page = case["kv_heads"], case["page"]
    group = case["q_heads"] // hk
    rows = _spread(case, case["rows_lo"], case["rows_hi"], case["sessions"], 0)
    ctx = _spread(case, case["ctx_lo"], case["ctx_hi"], case["sessions"], 1)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for i, (r, x) in enumerate(zip(rows, ctx)):
        n = x + r
        pages = s["table"][i, : -(-n // page)].long()
        known = (pages >= 0).repeat_interleave(page)[:n]
        known[x:] = True
        t = torch.arange(n, device="cuda")
        p = torch.arange(x, n, device="cuda")[:, None]
        seen = (t <= p) & known
        if case["window"]:
            seen &= (t < case["sinks"]) | (p - t < case["window"])
        for h in range(hk):
            keys = s["k"][0, pages.clamp(min=0), h].reshape(-1, case["head_dim"])[:n].double()
            values = s["v"][0, pages.clamp(min=0), h].reshape(-1, case["head_dim"])[:n].double()
            keys[x:] = s["k_new"][first: first + r, h].double()
            values[x:] = s["v_new"][first: first + r, h].double()
            for j in range(h * group, (h + 1) * group):
                score = s["q"][first: first + r, j].double() @ keys.T / math.sqrt(case["head_dim"])
                out[first: first + r, j] = torch.softmax(score.masked_fill(~seen, float("-inf")), -1) @ values
        first += r
    return {"out": out, "k": None, "v": None}
