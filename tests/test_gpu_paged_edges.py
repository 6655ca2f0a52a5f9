"""The paged cache's attention where its work is cut up: groups of heads that do not divide a tile, more tiles than
SMs, empty sessions between others, scores that keep rising, calls that share a workspace in graphs, and the binding's
checks of arguments.  References and tolerances as in test_gpu_paged."""
import numpy as np
import pytest

import paged_reference as ref

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_paged import Setup, gen, vc  # noqa: E402


def some(rows, n, seed=0):
    """(session, row) pairs: every session's first and last, and n more"""
    r = np.random.default_rng(seed)
    pairs = {(i, x) for i, m in enumerate(rows) if m for x in (0, m - 1)}
    full = [i for i, m in enumerate(rows) if m]
    return pairs | {(i, int(r.integers(rows[i]))) for i in r.choice(full, n)}


@pytest.mark.parametrize("heads,rows", [((6, 2, 64), [300, 1]), ((7, 1, 64), [150, 149]), ((6, 2, 128), [300, 1]),
                                        ((7, 1, 128), [75, 73]), ((32, 1, 64), [33, 2]), ((32, 1, 128), [17, 2]),
                                        ((100, 1, 128), [5, 2]), ((100, 1, 64), [11, 3]), ((256, 1, 64), [3, 5]),
                                        ((256, 1, 128), [3, 2]), ((300, 1, 64), [3, 1]), ((1, 1, 64), [513, 255]),
                                        ((3, 3, 128), [257, 256])], ids=str)
def test_groups_of_any_size(heads, rows):
    """whole tokens in a tile: groups that do not divide it, a token that fills it, one head (a tile of 512 tokens),
    groups beyond the tensor-core form's"""
    s = Setup(heads, 32, "bf16", 70, 5, [9, 90], rows, seed=3)
    out = s.run()
    s.check_appended()
    s.check(out, only=some(rows, 25))


@pytest.mark.parametrize("heads,page", [((16, 8, 64), 16), ((16, 8, 128), 64)])
def test_more_tiles_than_sms(heads, page):
    """some hundred pieces of work of very different lengths, sessions without rows in between"""
    r = np.random.default_rng(4)
    rows = [int(x) for x in r.integers(1, 260, 45)]
    for i in (0, 7, 8, 9, 44):
        rows[i] = 0
    ctx = [int(x) for x in r.integers(0, 400, 45)]
    s = Setup(heads, page, "fp16", 150, 9, ctx, rows, seed=5)
    for _ in range(2):     # the work counters are left as they were found
        out = s.run()
        s.check(out, only=some(rows, 40))


class Sessions(Setup):
    """Setup whose check looks up the sessions of `only` alone"""

    def check(self, out, only):
        full = self.ctx, self.rows, self.seqs, self.starts
        for i in sorted({i for i, _ in only}):
            a, n = int(full[3][i]), full[1][i]
            self.ctx, self.rows, self.seqs, self.starts = [full[0][i]], [n], [full[2][i]], np.array([a, a + n])
            super().check(out, only={(0, r) for j, r in only if j == i})
        self.ctx, self.rows, self.seqs, self.starts = full

    def parts(self, total=None):
        return super().parts(self.qkv.shape[0] - 5 if total is None else total)


@pytest.mark.parametrize("sessions", [60, 520])
def test_skipped_sessions_among_many_tiles(sessions):
    """tiles taken longest first (up to 512) or as the sessions come; sessions without a position, with one behind their
    length, and without rows change nothing for the others"""
    m = vc()
    r = np.random.default_rng(12)
    rows = [int(x) for x in r.integers(100, 300, sessions)] if sessions < 100 else [30] * sessions
    ctx = [int(x) for x in r.integers(0, 300, sessions)]
    rows[3] = rows[sessions - 1] = 0
    s = Sessions((16, 8, 64), 16, "bf16", 120, 3, ctx, rows, seed=13)
    pos = list(ctx)
    pos[1], pos[10], pos[20] = -1, ctx[10] + 1, -1
    out = s.run(pos=pos)
    assert int(s.cache.status) == m.VC_DEV_INVALID
    s.cache.status.zero_()
    for i in (1, 10, 20):
        part = out[s.starts[i]:s.starts[i + 1]]
        assert torch.equal(part, torch.full_like(part, 7.0))
    s.check(out, {p for p in some(rows, 40) if p[0] not in (1, 10, 20) and (p[0] < 30 or p[0] > sessions - 10)})


@pytest.mark.parametrize("batch", [1, 2, 40, 300])
def test_one_row_a_session_as_a_prompt(batch):
    """blocks of one row, in the prompts' form: as the frames' form gives them, within both forms' bounds"""
    ctx = [(37 * i) % 260 for i in range(batch)]
    s = Sessions((8, 2, 64), 16, "bf16", 100, 3, ctx, [1] * batch, seed=6)
    only = some([1] * batch, 20)
    s.check(s.run(), only)
    s.check(s.run(single=True), only)


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,step", [(t, s) for t in ("bf16", "fp16") for s in (0.25, 3.0)] + [("bf16", 40.0), ("fp16", 12.0)])
def test_scores_that_keep_rising(single, dtype, d, step):
    """every key scores higher than the last, by `step` in the exponent of 2: the running maximum moves within blocks,
    between them, or never by enough; and every other row the other way round.  (fp16 holds keys up to 65504: at 590
    positions and 128 dimensions a step of 0.6931 sqrt(128) 590 = 4627 for each unit, so 14 at most.)"""
    rows = [1, 1] if single else [90, 41]
    ctx = [500, 333]
    s = Setup((4, 2, d), 32, dtype, 0, 0, ctx, rows, seed=8)
    q, k, v = s.parts()
    q.zero_()
    q[::2, :, 0] = 1.0
    q[1::2, :, 0] = -1.0
    # the first dimension of key t is step ln 2 sqrt(d) t (as the type holds it): scores step ln 2 t
    for i, (c, n) in enumerate(zip(ctx, rows)):
        t = torch.arange(c + n, device="cuda", dtype=torch.float32) * (step * 0.6931 * d ** 0.5)
        page = s.table[s.seqs[i]].long()[torch.arange(c + n, device="cuda") // 32]
        s.k[0, page, :, torch.arange(c + n, device="cuda") % 32, 0] = t[:, None].to(s.k.dtype)
        k[int(s.starts[i]):int(s.starts[i]) + n, :, 0] = t[c:][:, None].to(s.k.dtype)
    s.check(s.run(single=single), only=some(rows, 20))


@pytest.mark.parametrize("heads", [(4, 2, 64), (4, 2, 128), (4, 2, 32)])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1), (2 ** 30, 5)])
def test_windows_and_sinks_of_any_size(heads, window, sinks):
    """as large as the type holds: every key up to the row's is seen; and the pages of a session stay"""
    s = Setup(heads, 16, "bf16", window, sinks, [300, 0], [140, 200], seed=10)
    s.check(s.run(), only=some([140, 200], 10))
    f = Setup(heads, 16, "bf16", window, sinks, [300, 0], [1, 1], seed=10)
    f.check(f.run(single=True))
    before = f.table.clone()
    f.cache.resize(add=1)
    assert torch.equal(f.table[before >= 0], before[before >= 0]) and f.lens.tolist() == [302, 2]


def test_two_graphs_that_share_a_workspace():
    """a prompt's graph and a frame's over one cache, replayed in turn, eager calls in between"""
    s = Setup((8, 2, 64), 16, "bf16", 90, 4, [700, 1300, 20], [60, 1, 33], seed=7)
    f = Setup((8, 2, 64), 16, "bf16", 90, 4, [500, 40, 2100], [1, 1, 1], seed=8)
    work = max(s.cache, f.cache, key=lambda c: c.c.workspace_bytes)
    for x in (s, f):
        x.cache.c.workspace, x.cache.c.workspace_bytes = work.c.workspace, work.c.workspace_bytes
    outs = [torch.zeros((x.starts[-1], 8, 64), dtype=torch.bfloat16, device="cuda") for x in (s, f)]
    args = []
    for x, single in ((s, False), (f, True)):
        i32 = dict(dtype=torch.int32, device="cuda")
        args.append((torch.tensor(x.ctx, **i32), None if single else torch.from_numpy(x.starts).cuda()))
    graphs = []
    for x, out, (pos, cu) in zip((s, f), outs, args):
        x.cache.attend(0, *x.parts(), out, pos, cu_rows=cu)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.cache.attend(0, *x.parts(), out, pos, cu_rows=cu)
        graphs.append(g)
    want = [o.clone() for o in outs]
    s.check(want[0])
    f.check(want[1])
    for turn in range(6):
        for o in outs:
            o.zero_()
        for g in (graphs if turn % 2 else graphs[::-1]):
            g.replay()
        if turn == 3:
            s.run()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_results_do_not_vary_from_call_to_call():
    """prompts and frames whose keys are split among CTAs: joined in a fixed order"""
    s = Setup((8, 2, 128), 64, "bf16", 0, 0, [6000], [40], seed=9)
    f = Setup((8, 2, 64), 64, "fp16", 0, 0, [9000, 3], [1, 1], seed=9)
    for x, single in ((s, False), (f, True)):
        first = x.run(single=single)
        for _ in range(10):
            assert torch.equal(x.run(single=single), first)


def test_page_calls_on_another_stream():
    m = vc()
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = m.PagedCache.empty(layers=2, pages=64, page_size=16, kv_heads=2, head_dim=32, seqs=4, columns=20, q_heads=4)
    pos, done, live = torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
    seqs = torch.tensor([2], **i32)
    lens, src, dst = torch.tensor([100], **i32), torch.tensor([2], **i32), torch.tensor([0], **i32)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    cache.resize(seqs, lens=lens, pos=pos, stream=st)
    cache.fork(src, dst, done=done, stream=st)
    cache.compact(live=live, stream=st)
    st.synchronize()
    assert pos.tolist() == [0] and done.tolist() == [1] and live.tolist() == [8]
    assert cache.lens.tolist() == [100, 0, 100, 0] and int((cache.refs == 2).sum()) == 6


def test_the_binding_checks_its_arguments():
    m = vc()
    i32 = dict(dtype=torch.int32, device="cuda")
    new = lambda **kw: m.PagedCache.empty(**{**dict(layers=2, pages=8, page_size=16, kv_heads=2, head_dim=32, seqs=3,  # noqa: E731
                                                    columns=4, q_heads=4), **kw})
    c = new()
    for kw in (dict(page_size=24), dict(head_dim=48), dict(q_heads=5), dict(window=-1), dict(sinks=-2)):
        with pytest.raises(m.VcError):
            new(**kw)
    with pytest.raises(ValueError):
        new(dtype=torch.float32)
    with pytest.raises(ValueError):
        m.PagedCache(c.k, c.v[:, :4], c.table, c.lens, c.refs, q_heads=4)
    with pytest.raises(ValueError):
        m.PagedCache(c.k, c.v, c.table, c.lens[:2], c.refs, q_heads=4)
    with pytest.raises(ValueError):
        m.PagedCache(c.k, c.v, c.table.long(), c.lens, c.refs, q_heads=4)
    with pytest.raises(ValueError):
        m.PagedCache(c.k, c.v, c.table, c.lens.cpu(), c.refs, q_heads=4)
    with pytest.raises(ValueError):
        m.PagedCache(c.k.transpose(2, 3), c.v, c.table, c.lens, c.refs, q_heads=4)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros((3, 4, 32), **bf), torch.zeros((3, 2, 32), **bf)
    pos = torch.zeros(3, **i32)
    good = (q, k, k.clone(), torch.zeros_like(q), pos)
    for at, bad in ((0, q.half()), (0, q[:, :3]), (0, q[:2]), (1, k[:2]), (1, None), (2, None), (3, q.float()), (3, q[:, :, :16]),
                    (0, q.transpose(1, 2).contiguous().transpose(1, 2)), (4, pos.long()), (4, pos.cpu()), (0, q.cpu())):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError):
            c.attend(0, *args)
    with pytest.raises(m.VcError):
        c.attend(2, *good)
    with pytest.raises(m.VcError):
        c.attend(0, q[:2], k[:2], k[:2], q[:2].clone(), pos)          # rows and sessions of unequal number
    with pytest.raises(ValueError):
        c.attend(0, *good, cu_rows=torch.zeros(3, **i32))
    with pytest.raises(ValueError):
        c.attend(0, *good, seqs=torch.zeros(2, **i32))
    with pytest.raises(m.VcError):
        c.attend(0, *good, scale=float("nan"))
    with pytest.raises(ValueError):
        c.resize(torch.zeros(2, **i32), lens=torch.zeros(3, **i32))
    with pytest.raises(ValueError):
        c.resize(add=1, pos=torch.zeros(2, **i32))
    with pytest.raises(m.VcError):
        c.resize(torch.zeros(4, **i32), add=1)
    with pytest.raises(ValueError):
        c.fork(torch.zeros(1, **i32), torch.zeros(2, **i32))
    with pytest.raises(ValueError):
        c.fork(torch.zeros(1, **i32), torch.ones(1, **i32), parts=m.session_parts([torch.zeros((2, 4), device="cuda")]))
    with pytest.raises(ValueError):
        m.session_parts([torch.zeros((2, 3, 4))])
    with pytest.raises(ValueError):
        m.session_parts([torch.zeros((2, 3, 4), device="cuda").transpose(0, 2)])
    with pytest.raises(ValueError):
        m.session_parts([torch.zeros((3,), device="cuda")] * 9)
    with pytest.raises(ValueError):
        m.session_parts([torch.zeros((3, 4), device="cuda"), torch.zeros((2, 5), device="cuda")])
    with pytest.raises(m.VcError):      # parts of 2 bytes a session
        c.fork(torch.zeros(1, **i32), torch.ones(1, **i32), parts=m.session_parts([torch.zeros((1, 3), **bf)]))
    with pytest.raises(ValueError):
        c.compact(live=torch.zeros(2, **i32))
    assert int(c.lens.sum()) == 0 and int(c.refs.sum()) == 0 and int(c.status) == 0


def test_appending_keeps_the_rest_of_a_page():
    """only the rows' own positions are written, in every form"""
    for rows, single in (([1, 1], True), ([7, 90], False)):
        s = Setup((8, 2, 64), 32, "bf16", 0, 0, [45, 17], rows, seed=11)
        before = s.k.clone(), s.v.clone()
        s.run(single=single)
        touched = torch.zeros((s.k.shape[1], 32), dtype=torch.bool)
        for i, (c, r) in enumerate(zip(s.ctx, s.rows)):
            row = s.table.cpu()[s.seqs[i]]
            for p in range(c, c + r):
                touched[row[p // 32], p % 32] = True
        for now, old in zip((s.k, s.v), before):
            same = (now == old).all(-1)[0].all(1).cpu()      # [pages][page], over the heads
            assert bool(same[~touched].all())
        s.check_appended()


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_a_session_read_twice_in_one_call(single, d):
    """without new rows a session may be named again: its rows at two places, each as alone"""
    rows = [1, 1] if single else [50, 33]
    s = Setup((8, 2, d), 32, "bf16", 60, 3, [200, 90], rows, seed=14)
    s.run(single=single)
    q = s.parts()[0]
    i32 = dict(dtype=torch.int32, device="cuda")
    want = s.run(append=False, single=single)
    twice = torch.cat([q[:rows[0]], q[:rows[0]]])
    out = torch.zeros_like(twice)
    cu = None if single else torch.tensor([0, rows[0], 2 * rows[0]], **i32)
    s.cache.attend(0, twice, None, None, out, torch.tensor([200, 200], **i32), seqs=torch.tensor([0, 0], **i32), cu_rows=cu)
    assert int(s.cache.status) == 0
    # each of the two is off by at most 2^-8 of sum w |v| (weights in bf16), 2^-8 of its value (rounded once) and, with a
    # 16th on top, the sums in fp32
    tol = 2 * 2.0 ** -8 * (float(s.v.float().abs().max()) + float(want.float().abs().max())) * 17 / 16
    assert float((out[:rows[0]].float() - want[:rows[0]].float()).abs().max()) <= tol
    assert float((out[rows[0]:].float() - want[:rows[0]].float()).abs().max()) <= tol


def test_two_caches_on_two_streams():
    """prompts and frames of caches with workspaces of their own, at the same time"""
    a = Setup((8, 2, 64), 16, "bf16", 150, 4, [700, 1300], [260, 133], seed=15)
    b = Setup((8, 2, 128), 32, "fp16", 0, 0, [900, 2100, 5], [1, 1, 1], seed=16)
    want = a.run(), b.run(single=True)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            a.run(out=outs[0])
        with torch.cuda.stream(streams[1]):
            b.run(single=True, out=outs[1])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
