"""The paged KV cache on the GPU: windowed attention with sinks against its definition in 64 bits, the page calls
against plain Python bookkeeping, and runs of them together."""
import numpy as np
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def vc():
    import attention_frame_decode_b200 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Setup:
    """a cache whose sessions hold ctx positions of random keys and values in pages of random order, and new rows"""

    def __init__(self, heads, page, dtype, window, sinks, ctx, rows, seed=0, spare=3, seqs=None, poison=False, layers=1):
        self.hq, self.hk, self.d = heads
        self.page, self.window, self.sinks, self.dtype = page, window, sinks, dtype
        self.ctx, self.rows = list(ctx), list(rows)
        n = len(self.ctx)
        self.seqs = list(range(n)) if seqs is None else list(seqs)
        n_seqs = max(self.seqs) + 1 + (0 if seqs is None else 2)
        g = gen(seed)
        lens = [c + r for c, r in zip(self.ctx, self.rows)]
        cols = max(-(-m // page) for m in lens) + 1
        used = sum(-(-m // page) for m in lens)
        pages = used + spare
        shape = (layers, pages, self.hk, page, self.d)
        dt = DT[dtype]
        self.k = torch.randn(shape, generator=g, device="cuda").to(dt)
        self.v = torch.randn(shape, generator=g, device="cuda").to(dt)
        order = torch.randperm(pages, generator=g, device="cuda").cpu().tolist()
        table = np.full((n_seqs, cols), -1, np.int32)
        refs = np.zeros(pages, np.int32)
        full = np.zeros(n_seqs, np.int32)
        at = 0
        for s, m in zip(self.seqs, lens):
            for c in range(-(-m // page)):
                table[s, c] = order[at]
                refs[order[at]] = 1
                at += 1
            full[s] = m
        self.table, self.refs, self.lens = (torch.from_numpy(x).cuda() for x in (table, refs, full))
        total = sum(self.rows)
        self.qkv = torch.randn((total + 5, (self.hq + 2 * self.hk) * self.d), generator=g, device="cuda").to(dt)
        if poison:   # everything that no query of the call may see
            for t in (self.k, self.v):
                for s, c, r in zip(self.seqs, self.ctx, self.rows):
                    for p in range(-(-(c + r) // page) * page):
                        hidden = p >= c + r or (window and sinks <= p <= c - window)
                        if hidden:
                            t[0, table[s, p // page], :, p % page] = float("nan") if p % 2 else float("inf")
                for f in np.nonzero(refs == 0)[0]:
                    t[0, f] = float("nan")
        self.cache = vc().PagedCache(self.k, self.v, self.table, self.lens, self.refs, q_heads=self.hq, window=window,
                                     sinks=sinks)
        self.starts = np.concatenate([[0], np.cumsum(self.rows)]).astype(np.int32)

    def parts(self, total=None):
        total = self.starts[-1] if total is None else total
        hq, hk, d = self.hq, self.hk, self.d
        x = self.qkv[:total]
        return (x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                x[:, (hq + hk) * d:].unflatten(1, (hk, d)))

    def run(self, total=None, append=True, single=False, scale=0.0, pos=None, stream=None, out=None):
        q, k, v = self.parts(total)
        if out is None:
            out = torch.full((q.shape[0], self.hq, self.d), 7.0, dtype=q.dtype, device="cuda")
        pos = torch.tensor(self.ctx if pos is None else pos, dtype=torch.int32, device="cuda")
        seqs = torch.tensor(self.seqs, dtype=torch.int32, device="cuda")
        cu = None if single else torch.from_numpy(self.starts).cuda()
        self.cache.attend(0, q, k if append else None, v if append else None, out, pos, seqs=seqs, cu_rows=cu, scale=scale,
                          stream=stream)
        return out

    def history(self, i, v=False):
        """[positions][heads][dims] of session i from the pool"""
        pool = (self.v if v else self.k)[0].float().cpu().numpy()
        row = self.table.cpu().numpy()[self.seqs[i]]
        m = self.ctx[i] + self.rows[i]
        x = np.stack([pool[max(row[p // self.page], 0), :, p % self.page] for p in range(m)])
        return x

    def check(self, out, scale=None, mapped=None, only=None):
        """every row (or `only` (session, row) pairs) against the definition"""
        scale = ref.default_scale(self.d) if scale is None else scale
        got = out.float().cpu().numpy()
        q = self.parts()[0].float().cpu().numpy()
        worst = 0.0
        for i, (c, r) in enumerate(zip(self.ctx, self.rows)):
            keys, values = self.history(i), self.history(i, v=True)
            for nth in range(r):
                if only is not None and (i, nth) not in only:
                    continue
                seen = ref.seen_keys(c + nth, c + r, self.window, self.sinks)
                if mapped is not None:
                    seen &= mapped(i, np.arange(c + r))
                for h in range(self.hq):
                    j = h * self.hk // self.hq
                    o, a, s, av = ref.attend_row(q[self.starts[i] + nth, h], keys[:, j], values[:, j], seen, scale)
                    tol = ref.tolerance(o, a, s, av, self.d, ref.HALF_STEP[self.dtype], ref.FLOOR[self.dtype])
                    err = np.abs(got[self.starts[i] + nth, h] - o)
                    assert np.all(err <= tol), (i, nth, h, float(err.max()), float(tol[err.argmax()]))
                    worst = max(worst, float((err / tol).max()))
        assert int(self.cache.status) == 0
        return worst

    def check_appended(self):
        k, v = (x.cpu() for x in self.parts()[1:])
        for i, (c, r) in enumerate(zip(self.ctx, self.rows)):
            for t, new in ((self.k, k), (self.v, v)):
                row = self.table.cpu()[self.seqs[i]]
                for nth in range(r):
                    p = c + nth
                    assert torch.equal(t[0, row[p // self.page], :, p % self.page].cpu(), new[self.starts[i] + nth])


# ---- single frames ------------------------------------------------------------------------------

FRAMES = [
    # heads, page, dtype, window, sinks, ctx
    ((40, 8, 128), 64, "bf16", 1024, 4, [2000]),
    ((40, 8, 128), 64, "bf16", 0, 0, [0, 1, 63, 64, 65, 700]),
    ((8, 2, 32), 16, "fp16", 100, 3, [0, 15, 16, 99, 100, 101, 102, 103, 517]),
    ((8, 2, 32), 16, "bf16", 1, 0, [0, 31, 32, 200]),
    ((8, 2, 32), 128, "fp16", 1, 1, [0, 127, 128, 300]),
    ((32, 8, 64), 32, "fp16", 300, 17, [5, 31, 299, 300, 301, 316, 317, 1200]),
    ((16, 4, 64), 256, "bf16", 64, 200, [10, 199, 200, 263, 264, 265, 1000]),
    ((8, 4, 256), 16, "bf16", 333, 20, [7, 400, 1111]),
    ((8, 4, 256), 64, "fp16", 0, 9, [3, 640]),
    ((5, 1, 128), 32, "bf16", 5, 500, [1, 499, 500, 505, 506, 900]),
    ((12, 12, 64), 16, "bf16", 77, 0, [50, 77, 300]),
    ((16, 1, 128), 64, "bf16", 500, 64, [33, 1500]),
    ((34, 2, 64), 64, "fp16", 129, 5, [128, 129, 130, 800]),     # 17 query heads to a KV head
    ((48, 1, 32), 16, "bf16", 0, 0, [40, 350]),                  # 48
]


@pytest.mark.parametrize("heads,page,dtype,window,sinks,ctx", FRAMES, ids=str)
def test_frames_match_the_definition(heads, page, dtype, window, sinks, ctx):
    s = Setup(heads, page, dtype, window, sinks, ctx, [1] * len(ctx), seed=len(ctx))
    out = s.run(single=True)
    s.check_appended()
    s.check(out)


@pytest.mark.parametrize("heads,page,dtype,window,sinks,ctx", FRAMES[:8], ids=str)
def test_frames_are_not_touched_by_what_they_do_not_see(heads, page, dtype, window, sinks, ctx):
    s = Setup(heads, page, dtype, window, sinks, ctx, [1] * len(ctx), seed=3, poison=True)
    s.check(s.run(single=True))


def test_frames_of_listed_sessions_and_without_new_rows():
    s = Setup((32, 8, 64), 32, "bf16", 200, 8, [150, 3, 420], [1, 1, 1], seqs=[4, 0, 2])
    out = s.run(single=True)
    s.check_appended()
    s.check(out)
    again = s.run(single=True, append=False)
    assert torch.equal(out, again)


def test_frames_of_many_sessions():
    rng = np.random.default_rng(5)
    ctx = [int(x) for x in rng.integers(0, 900, 130)]
    s = Setup((8, 2, 32), 16, "bf16", 250, 5, ctx, [1] * len(ctx))
    s.check(s.run(single=True))


def test_long_frames_split_over_the_keys():
    s = Setup((5, 1, 128), 64, "bf16", 0, 0, [30011, 4], [1, 1])
    s.check(s.run(single=True))
    s = Setup((8, 2, 32), 128, "fp16", 20000, 700, [25013], [1])
    s.check(s.run(single=True))


@pytest.mark.parametrize("scale", [0.5, -0.125, 1e-30, 30.0])
def test_scale(scale):
    # 30: scores of some hundreds, weights that underflow
    s = Setup((8, 2, 64), 32, "fp16", 0, 0, [120, 3], [1, 1])
    s.check(s.run(single=True, scale=scale), scale=scale)


# ---- prompts ------------------------------------------------------------------------------------

PROMPTS = [
    ((8, 2, 32), 16, "fp16", 100, 3, [0], [257]),
    ((40, 8, 128), 64, "bf16", 96, 4, [0, 40], [130, 27]),
    ((40, 8, 128), 64, "bf16", 0, 0, [200, 0, 65], [1, 2, 64]),
    ((32, 8, 64), 32, "bf16", 128, 16, [0, 500, 127, 31], [33, 1, 129, 64]),
    ((16, 4, 64), 128, "fp16", 0, 0, [0, 300], [150, 40]),
    ((8, 4, 256), 16, "bf16", 60, 70, [0, 100], [90, 65]),
    ((12, 12, 64), 16, "fp16", 1, 0, [0, 5], [70, 70]),
    ((5, 1, 128), 256, "fp16", 200, 300, [0, 250], [260, 131]),
    ((48, 1, 32), 16, "bf16", 64, 1, [0], [100]),
    ((2, 2, 128), 32, "bf16", 500, 10, [0], [700]),
    ((2, 1, 64), 16, "fp16", 0, 0, [1000], [300]),
]


@pytest.mark.parametrize("heads,page,dtype,window,sinks,ctx,rows", PROMPTS, ids=str)
def test_prompts_match_the_definition(heads, page, dtype, window, sinks, ctx, rows):
    s = Setup(heads, page, dtype, window, sinks, ctx, rows, seed=1)
    out = s.run()
    s.check_appended()
    s.check(out)


@pytest.mark.parametrize("heads,page,dtype,window,sinks,ctx,rows", PROMPTS[:8], ids=str)
def test_prompts_are_not_touched_by_what_they_do_not_see(heads, page, dtype, window, sinks, ctx, rows):
    s = Setup(heads, page, dtype, window, sinks, ctx, rows, seed=2, poison=True)
    s.check(s.run())


@pytest.mark.parametrize("heads,dtype", [((4, 2, 128), "bf16"), ((4, 2, 64), "fp16"), ((4, 1, 32), "bf16"), ((2, 1, 256), "fp16")])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_value_that_is_not_finite_reaches_only_the_rows_that_see_it(heads, dtype, value):
    s = Setup(heads, 32, dtype, 60, 2, [0], [200], seed=4)
    hq, hk, d = heads
    bad = 77
    s.parts()[2][bad, 0, 3] = value                 # dimension 3 of the first KV head's value
    out = s.run()
    clean = Setup(heads, 32, dtype, 60, 2, [0], [200], seed=4)
    clean.run()
    rows = [(0, r) for r in range(200) if not bad <= r < bad + 60]
    s.check(out, only=set(rows[:40] + rows[-40:]))
    got = out.float()
    hit = got[bad:bad + 60, : hq // hk, 3]
    assert not torch.isfinite(hit).any()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[bad:bad + 60, : hq // hk, 3] = False
    assert torch.isfinite(got[rest]).all()
    s2 = Setup(heads, 32, dtype, 60, 2, [0], [200], seed=4)
    s2.parts()[1][bad, 0, 5] = value                # and a key's: its weight is not a number for who sees it
    got = s2.run().float()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[bad:bad + 60, : hq // hk] = False
    assert torch.isfinite(got[rest]).all()


def test_blocks_of_a_prompt_give_the_whole_prompts_rows():
    """a prompt handed in block by block: every row sees the same keys as in one call"""
    whole = Setup((8, 2, 64), 32, "bf16", 90, 7, [0], [300], seed=9)
    all_rows = whole.run()
    cuts = [0, 1, 34, 160, 161, 300]
    s = Setup((8, 2, 64), 32, "bf16", 90, 7, [0], [300], seed=9)
    q, k, v = s.parts()
    for a, b in zip(cuts, cuts[1:]):
        out = torch.empty((b - a, 8, 64), dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        s.cache.attend(0, q[a:b], k[a:b], v[a:b], out, torch.tensor([a], dtype=torch.int32, device="cuda"), cu_rows=cu)
        all_rows[a:b] = out
    whole.check(all_rows)


@pytest.mark.parametrize("single", [True, False])
def test_rows_without_a_key_are_zero(single):
    """a session whose pages are not in the table: nothing to see, and nothing is written"""
    rows = [1, 1] if single else [70, 3]
    s = Setup((8, 2, 64), 16, "bf16", 30, 4, [40, 9], rows)
    keep = s.k.clone()
    s.table.fill_(-1)
    out = s.run(single=single)
    assert torch.equal(out, torch.zeros_like(out)) and torch.equal(s.k, keep) and int(s.cache.status) == 0


def test_holes_in_the_table():
    s = Setup((8, 2, 64), 16, "fp16", 0, 0, [100, 250], [1, 1], seed=6)
    t = s.table.cpu().numpy()
    gone = {0: {0, 3}, 1: {2, 3, 4, 5, 9}}
    for i, cols in gone.items():
        for c in cols:
            s.table[i, c] = -1 if c % 2 else 1 << 20      # out of range counts as none
    mapped = lambda i, p: ~np.isin(p // 16, list(gone[i]))  # noqa: E731
    out = s.run(single=True)
    hist = (s.table.clone(), s.table.copy_(torch.from_numpy(t)))
    s.check(out, mapped=mapped)
    del hist


@pytest.mark.parametrize("single", [True, False])
def test_skipped_sessions_and_rows_behind_the_last(single):
    m = vc()
    rows = [1, 1, 1] if single else [40, 5, 80]
    s = Setup((8, 2, 64), 16, "bf16", 50, 4, [20, 9, 33], rows)
    before = s.k.clone()
    # session 1 is skipped, session 2 names a position behind its length
    total = 3 if single else s.starts[-1] + 5
    out = s.run(total=total, single=single, pos=[20, -1, 34])
    assert int(s.cache.status) == m.VC_DEV_INVALID
    s.cache.status.zero_()
    a, b = s.starts[1], s.starts[3]
    assert torch.equal(out[a:], torch.full_like(out[a:], 7.0))
    row = s.table.cpu()
    for i in (1, 2):
        for e in row[i][row[i] >= 0]:
            assert torch.equal(s.k[0, e], before[0, e])
    s.check(out, only={(0, r) for r in range(rows[0])})


def test_bad_indices_are_reported_and_skipped():
    m = vc()
    s = Setup((8, 2, 64), 16, "bf16", 50, 4, [20, 9], [3, 2])
    q, k, v = s.parts()
    i32 = dict(dtype=torch.int32, device="cuda")
    keep = s.k.clone()

    def call(seqs, cu, pos):
        s.cache.status.zero_()
        out = torch.full((5, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        s.cache.attend(0, q, k, v, out, torch.tensor(pos, **i32), seqs=torch.tensor(seqs, **i32), cu_rows=torch.tensor(cu, **i32))
        return out, int(s.cache.status)

    for seqs, cu, pos in (([-1, 7], [0, 3, 5], [20, 9]), ([0, 1], [0, 3, 5], [1 << 30, 1 << 30]), ([0, 1], [3, 0, -4], [20, 9]),
                          ([0, 1], [0, 1 << 30, 1 << 30], [20, 9]), ([0, 1], [-3, 0, 0], [20, 9])):
        out, status = call(seqs, cu, pos)
        assert status == m.VC_DEV_INVALID, (seqs, cu, pos)
        assert torch.equal(out, torch.full_like(out, 7.0)) and torch.equal(s.k, keep)


def test_pool_offsets_beyond_32_bits():
    """pages behind 2^31 elements and behind 2^32 bytes; only the touched pages are written"""
    hk, page, d, pages = 8, 128, 128, 16400            # 2.15e9 elements a pool
    k = torch.empty((1, pages, hk, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 31
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 5], [pages - 2, pages - 7, 8]], **i32)
    refs = torch.zeros(pages, **i32)
    g = gen(1)
    for e in table.flatten().tolist():
        k[0, e] = torch.randn((hk, page, d), generator=g, device="cuda")
        v[0, e] = torch.randn((hk, page, d), generator=g, device="cuda")
        refs[e] = 1
    for rows, single in (([1, 1], True), ([60, 2], False)):
        s = Setup((8, 8, 128), page, "bf16", 200, 4, [300, 290], rows)
        s.k, s.v, s.table, s.lens = k, v, table, torch.tensor([300 + rows[0], 290 + rows[1]], **i32)
        s.cache = vc().PagedCache(k, v, table, s.lens, refs, q_heads=8, window=200, sinks=4)
        s.history = lambda i, v=False, s=s: _gather(s, i, v)
        s.check(s.run(single=single), only={(0, 0), (0, rows[0] - 1), (1, rows[1] - 1)})


def _gather(s, i, values):
    pool = (s.v if values else s.k)[0]
    m = s.ctx[i] + s.rows[i]
    p = torch.arange(m, device="cuda")
    return pool[s.table[i].long()[p // s.page], :, p % s.page].float().cpu().numpy()


# ---- streams and graphs ---------------------------------------------------------------------------


def test_attend_on_another_stream():
    s = Setup((40, 8, 128), 64, "bf16", 300, 4, [700, 20], [1, 1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.full((2, 40, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        s.run(single=True, out=out)
    st.synchronize()
    s.check(out)
    s.run(single=True, out=out, stream=st)
    st.synchronize()
    s.check(out)


def test_a_frame_in_a_graph():
    """resize by one and attend, captured once and replayed: every replay is the next frame"""
    m = vc()
    g = gen(2)
    i32 = dict(dtype=torch.int32, device="cuda")
    hq, hk, d, page, window, sinks = 8, 2, 64, 16, 40, 3
    cache = m.PagedCache.empty(layers=1, pages=40, page_size=page, kv_heads=hk, head_dim=d, seqs=2, columns=20, q_heads=hq,
                               window=window, sinks=sinks)
    x = torch.randn((120, 2, (hq + 2 * hk) * d), generator=g, device="cuda").to(torch.bfloat16)
    row, pos = torch.zeros_like(x[0]), torch.zeros(2, **i32)
    out = torch.zeros((2, hq, d), dtype=torch.bfloat16, device="cuda")
    q, k, v = row[:, :hq * d].unflatten(1, (hq, d)), row[:, hq * d:-hk * d].unflatten(1, (hk, d)), row[:, -hk * d:].unflatten(1, (hk, d))

    def frame():
        cache.resize(add=1, pos=pos)
        cache.attend(0, q, k, v, out, pos)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        row.copy_(x[0])
        frame()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        frame()
    for t in range(1, 120):
        row.copy_(x[t])
        graph.replay()
        if t % 17 == 0 or t == 119:
            h = x[: t + 1].float().cpu().numpy()
            for b in range(2):
                seen = ref.seen_keys(t, t + 1, window, sinks)
                for head in (0, hq - 1):
                    j = head * hk // hq
                    keys = h[:, b, (hq + j) * d:(hq + j + 1) * d]
                    vals = h[:, b, (hq + hk + j) * d:(hq + hk + j + 1) * d]
                    o, a, sc, av = ref.attend_row(h[t, b, head * d:(head + 1) * d], keys, vals, seen, ref.default_scale(d))
                    tol = ref.tolerance(o, a, sc, av, d, ref.HALF_STEP["bf16"], ref.FLOOR["bf16"])
                    assert np.all(np.abs(out[b, head].float().cpu().numpy() - o) <= tol), (t, b, head)
    assert cache.lens.tolist() == [120, 120] and int(cache.status) == 0
    # the window's pages and the sinks' only
    assert int((cache.refs > 0).sum()) <= 2 * (1 + window // page + 2)


# ---- page calls -----------------------------------------------------------------------------------


class Pair:
    """a cache beside its plain bookkeeping; page contents are followed position by position"""

    def __init__(self, pages, page, seqs, columns, window=0, sinks=0, layers=2, hk=2, d=32):
        self.book = ref.Book(pages, page, seqs, columns, window, sinks)
        self.cache = vc().PagedCache.empty(layers=layers, pages=pages, page_size=page, kv_heads=hk, head_dim=d, seqs=seqs,
                                           columns=columns, q_heads=hk, window=window, sinks=sinks, dtype=torch.float16)
        g = gen(pages)
        self.cache.k.copy_(torch.randn(self.cache.k.shape, generator=g, device="cuda"))
        self.cache.v.copy_(torch.randn(self.cache.v.shape, generator=g, device="cuda"))
        self.k, self.v = self.cache.k.cpu().clone(), self.cache.v.cpu().clone()

    def _same(self):
        b, c = self.book, self.cache
        for src, dst, n in b.copies:
            for t in (self.k, self.v):
                t[:, dst, :, :n] = t[:, src, :, :n]
        b.copies.clear()
        assert c.table.tolist() == b.table
        assert c.lens.tolist() == b.len
        assert c.refs.tolist() == b.refs
        assert int(c.status) == b.status
        assert torch.equal(c.k.cpu(), self.k) and torch.equal(c.v.cpu(), self.v)

    def resize(self, seqs, targets, add=0):
        pos = torch.full((len(targets),), 99, dtype=torch.int32, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cache.resize(seqs=None if seqs is None else i32(seqs), lens=i32(targets), add=add, pos=pos)
        want = self.book.resize(list(range(len(targets))) if seqs is None else seqs, [t + add for t in targets])
        assert pos.tolist() == want
        self._same()
        return want

    def fork(self, src, dst, parts=None):
        done = torch.full((len(src),), 99, dtype=torch.int32, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cache.fork(i32(src), i32(dst), parts=parts, done=done)
        want = self.book.fork(src, dst)
        assert done.tolist() == want
        self._same()
        return want

    def compact(self):
        live = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cache.compact(live=live)
        n, moves = self.book.compact()
        for a, b in moves:
            for t in (self.k, self.v):
                t[:, b] = t[:, a]
        assert live.tolist() == [n]
        self._same()
        return n


def test_resize_by_hand():
    p = Pair(pages=9, page=16, seqs=4, columns=5, window=20, sinks=3)
    assert p.resize(None, [1, 16, 17, 0]) == [0, 0, 0, 0]
    assert p.resize([2, 0], [60, 16]) == [17, 1]
    assert p.resize([1, 1, 4, -1], [5, 6, 1, 1]) == [5, -1, -1, -1]               # twice, out of range
    assert p.resize([3], [-1]) == [-1]                                              # below 0
    assert p.resize([3], [81]) == [-1]                                              # more than the columns hold
    # more than is free, and so is what a later row asks for; a row that asks for none is served
    assert p.resize([3, 0, 1], [70, 17, 6]) == [-1, -1, 5]
    assert p.resize([2, 3], [60, 30], add=1) == [60, 0]
    assert p.resize([2, 1], [40, 3]) == [40, 3]                 # cut inside a page that it holds
    assert p.resize([2], [30]) == [-1]                          # and inside one that the window has given up
    assert p.resize(None, [0, 0, 0, 0]) == [0, 0, 0, 0]
    assert p.cache.refs.tolist() == [0] * 9


def test_window_gives_pages_back():
    p = Pair(pages=64, page=16, seqs=1, columns=64, window=33, sinks=17)
    for n in [1, 40, 41, 200, 201, 202, 215, 300, 640, 641, 1000, 1001]:
        assert p.resize(None, [n])[0] >= 0
    held = [c for c in range(64) if p.book.table[0][c] >= 0]
    assert held[:2] == [0, 1] and held[2] >= 40
    assert p.resize(None, [500]) == [-1]            # inside a page given up
    assert p.resize(None, [496]) == [496]           # at a page's border: what is left behind it are the sinks
    assert p.resize(None, [530]) == [496]
    assert p.resize(None, [20]) == [20] and p.resize(None, [0]) == [0]
    assert p.cache.refs.tolist() == [0] * 64


def test_fork_shares_and_copies_on_write():
    p = Pair(pages=30, page=16, seqs=6, columns=8, window=0)
    p.resize([0, 1], [40, 32])
    assert p.fork([0, 0, 1], [2, 3, 4]) == [1, 1, 1]
    p.resize([2, 3], [50, 41])
    p.resize([2], [20])                    # back into a page that session 0 shares
    p.resize([2, 0], [25, 45])             # writes there: a copy for session 2
    p.resize([4], [30])
    p.resize([4, 1], [31, 30])
    p.resize([1, 4], [33, 40])             # both leave the page that they share
    assert p.fork([0], [1]) == [1]         # onto a session that holds pages
    assert p.fork([5], [0]) == [1]         # an empty session
    assert p.fork([0, 2, 2, 3, 9, 3], [0, 4, 4, 2, 5, -1]) == [0, 1, 0, 0, 0, 0]
    p.resize(None, [0] * 6)
    assert p.cache.refs.tolist() == [0] * 30


def test_fork_without_a_free_page():
    p = Pair(pages=4, page=16, seqs=4, columns=4)
    p.resize([0, 1], [40, 16])
    # no page left for 2; nothing to copy for 3: no page needed; 1 is a source too: a bad row
    assert p.fork([0, 1, 0], [2, 3, 1]) == [0, 1, 0]
    assert p.fork([1, 2], [3, 0]) == [1, 1]              # 2 is empty, and so is 0 then


def test_compact_moves_the_fewest_pages():
    p = Pair(pages=50, page=16, seqs=8, columns=8)
    p.resize(None, [60, 100, 20, 5, 90, 128, 1, 33])
    p.resize([0, 2, 4], [0, 0, 0])
    p.fork([5, 5], [0, 2])
    assert p.compact() == sum(r > 0 for r in p.book.refs)
    p.resize([5], [3])
    p.compact()
    p.compact()
    p.resize(None, [0] * 8)
    assert p.compact() == 0


def test_compact_of_a_full_pool_and_over_chunks():
    p = Pair(pages=9000, page=16, seqs=3, columns=4096, layers=1, hk=1)
    assert p.resize(None, [16 * 4090, 16 * 4096, 16 * 814]) == [0, 0, 0]
    assert p.compact() == 9000
    p.resize([0], [16 * 3])
    p.compact()
    p.resize([1], [16 * 4000 + 1])
    p.compact()


@pytest.mark.parametrize("seed", range(6))
def test_page_calls_in_random_order(seed):
    rng = np.random.default_rng(seed)
    window = int(rng.choice([0, 1, 25, 80]))
    seqs = int(rng.integers(2, 40))
    p = Pair(pages=int(rng.integers(20, 160)), page=int(rng.choice([16, 32])), seqs=seqs, columns=12, window=window,
             sinks=int(rng.integers(0, 40)), layers=1)
    for _ in range(60):
        op = rng.integers(0, 8)
        n = int(rng.integers(1, seqs + 1))
        if op < 3:
            p.resize(None, [x + 1 for x in p.book.len])
        elif op < 5:
            who = [int(x) for x in rng.integers(0, seqs, n)]
            p.resize(who, [int(x) for x in rng.integers(0, 12 * p.book.page + 4, n)])
        elif op < 6:
            who = [int(x) for x in rng.permutation(seqs)[:n]]
            p.resize(who, [max(0, p.book.len[s] - int(rng.integers(0, 30))) for s in who])
        elif op < 7:
            p.fork([int(x) for x in rng.integers(-1, seqs, n)], [int(x) for x in rng.integers(0, seqs + 1, n)])
        else:
            p.compact()


def test_many_sessions_in_one_call():
    """more sessions than a CTA has threads, more pages than one pass over the counts takes"""
    n = 2500
    p = Pair(pages=40000, page=16, seqs=n, columns=40, window=100, sinks=5, layers=1, hk=1)
    rng = np.random.default_rng(0)
    p.resize(None, [int(x) for x in rng.integers(0, 300, n)])
    p.resize(None, [int(x) for x in rng.integers(1, 60, n)], add=300)
    order = [int(x) for x in rng.permutation(n)]
    p.fork(order[:1000], order[1000:2000])
    p.resize(order, [p.book.len[s] + 1 for s in order])
    p.compact()


def test_fork_copies_the_sessions_state():
    m = vc()
    p = Pair(pages=20, page=16, seqs=5, columns=4)
    p.resize([0, 1], [20, 50])
    g = gen(0)
    ssm = torch.randn((3, 5, 8, 16, 33), generator=g, device="cuda")            # 16-byte multiples
    big = torch.randn((2, 5, 70001), generator=g, device="cuda")                # not
    ring = torch.randn((2, 5, 4, 90), generator=g, device="cuda").to(torch.bfloat16)
    ctx = torch.arange(5, dtype=torch.int32, device="cuda")
    want = [t.clone() for t in (ssm, big, ring, ctx)]
    parts = m.session_parts([ssm, big, ring, ctx])
    assert p.fork([1, 0, 1, 9], [4, 2, 4, 3], parts=parts) == [1, 1, 0, 0]
    for t in want[:3]:
        t[:, 4], t[:, 2] = t[:, 1].clone(), t[:, 0].clone()
    want[3][4], want[3][2] = 1, 0
    for t, w in zip((ssm, big, ring, ctx), want):
        assert torch.equal(t, w)


# ---- all of it together ---------------------------------------------------------------------------


def test_sessions_from_an_opening_context_to_their_end():
    """one opening context, forked to callers who stream frame by frame past their window, one of them cut back,
    one ended, the pool drawn together in between; every output against the callers' own histories"""
    m = vc()
    hq, hk, d, page, window, sinks = 10, 2, 64, 16, 50, 6
    rng = np.random.default_rng(3)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = m.PagedCache.empty(layers=2, pages=60, page_size=page, kv_heads=hk, head_dim=d, seqs=5, columns=40, q_heads=hq,
                               window=window, sinks=sinks)
    hist = {s: [np.zeros((0, 2, hk, d), np.float32), np.zeros((0, 2, hk, d), np.float32)] for s in range(5)}

    def take(who, counts):
        """`counts` new rows for the sessions `who`, both layers"""
        total = sum(counts)
        pos = torch.zeros(len(who), **i32)
        seqs = torch.tensor(who, **i32)
        cache.resize(seqs, lens=torch.tensor([hist[s][0].shape[0] + c for s, c in zip(who, counts)], **i32), pos=pos)
        assert pos.tolist() == [hist[s][0].shape[0] for s in who]
        x = torch.from_numpy(rng.normal(size=(2, total, hq + 2 * hk, d)).astype(np.float32)).cuda().to(torch.bfloat16)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), **i32)
        out = torch.empty((2, total, hq, d), dtype=torch.bfloat16, device="cuda")
        for layer in range(2):
            cache.attend(layer, x[layer, :, :hq], x[layer, :, hq:hq + hk], x[layer, :, hq + hk:], out[layer], pos, seqs=seqs,
                         cu_rows=None if total == len(who) else cu)
        y, got = x.float().cpu().numpy(), out.float().cpu().numpy()
        row = 0
        for s, c in zip(who, counts):
            old = hist[s][0].shape[0]
            for w, lo in ((0, hq), (1, hq + hk)):
                hist[s][w] = np.concatenate([hist[s][w], y[:, row:row + c, lo:lo + hk].transpose(1, 0, 2, 3)])
            for nth in range(c):
                seen = ref.seen_keys(old + nth, old + c, window, sinks)
                for layer in range(2):
                    for h in range(0, hq, 3):
                        j = h * hk // hq
                        o, a, sc, av = ref.attend_row(y[layer, row + nth, h], hist[s][0][:, layer, j], hist[s][1][:, layer, j],
                                                      seen, ref.default_scale(d))
                        tol = ref.tolerance(o, a, sc, av, d, ref.HALF_STEP["bf16"], ref.FLOOR["bf16"])
                        assert np.all(np.abs(got[layer, row + nth, h] - o) <= tol), (s, nth, layer, h)
            row += c

    def fork(src, dst):
        cache.fork(torch.tensor(src, **i32), torch.tensor(dst, **i32))
        for a, b in zip(src, dst):
            hist[b] = [t.copy() for t in hist[a]]

    take([0], [75])
    fork([0, 0, 0], [1, 2, 4])
    for _ in range(30):
        take([4, 0, 2, 1], [1, 1, 1, 1])
    cache.compact()
    take([1, 2], [40, 1])
    n = hist[2][0].shape[0] - 3                              # the last three frames of session 2 taken back
    cache.resize(torch.tensor([2], **i32), lens=torch.tensor([n], **i32))
    hist[2] = [t[:n] for t in hist[2]]
    take([2, 4], [5, 1])
    cache.resize(torch.tensor([0], **i32), lens=torch.zeros(1, **i32))   # session 0 ends
    hist[0] = [t[:0] for t in hist[0]]
    fork([4], [3])
    cache.compact()
    for _ in range(20):
        take([3, 4, 1, 2], [1, 1, 1, 1])
    take([0], [33])
    cache.resize(lens=torch.zeros(5, **i32))
    assert int(cache.status) == 0 and cache.refs.tolist() == [0] * 60
