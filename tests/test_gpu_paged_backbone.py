"""The backbone over a paged cache: prefill and frames whose attention layers keep their keys and values in pages.

Where the window covers the context, the whole stack is held to the oracle exactly as over the state's own rows (the
bounds of the decode and prefill tests).  Where it does not, an attention layer is held to its equations in 64 bits, on
the residual stream that entered it and the keys and values in its pages, within the bound of WindowedLayer; every test
checks that the unwindowed layer is more than five times that bound away.
"""
import numpy as np
import pytest

import mirror_layer
import oracle
import synth
from paged_reference import CAPACITY, FLOOR, HALF_STEP, INVALID, attend_row, default_scale, seen_keys, tolerance
from test_gpu_decode import Run, check_step, nano_layer_cfg
from test_gpu_prefill import PrefillRun

TOL = 2e-2

pytestmark = pytest.mark.gpu


def bits(x):
    import torch
    return torch.from_numpy(x).cuda().view(torch.bfloat16)


def i32(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class PagedRun(Run):
    """Run whose backbone steps over a paged cache (the state has no rows of its own)"""

    def __init__(self, cfg, seed, B, cap, page=16, window=0, sinks=0, pages=None, columns=None, slots=None, taps=True):
        super().__init__(cfg, seed, B, cap, taps=taps)
        columns = columns or -(-cap // page)
        self.st = self.dm.new_state(B, 0)
        self.cache = self.bb.new_cache(pages or B * columns, page, columns, window, sinks)

    def step(self, t, slots=None, x=None):
        import torch
        x = synth.frame_inputs(self.cfg, self.seed, t, self.B) if x is None else x
        sl = None if slots is None else i32(slots)
        self.bb.step_paged(bits(x), self.st, self.cache, self.tt, self.tf, slots=sl)
        torch.cuda.synchronize()
        return self.om.step(self.ost, x, oracle.MIRROR, slots=slots, taps=True)


@pytest.mark.parametrize("graph", [0, 1])
@pytest.mark.parametrize("wfmt,B,frames", [(synth.FMT_W8, 1, 64), (synth.FMT_BF16, 3, 20), (synth.FMT_W4, 2, 20),
                                           (synth.FMT_W3, 12, 6)])
def test_frames_match_the_oracle(cuda, wfmt, B, frames, graph):
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config(wfmt=wfmt, head_fmt=wfmt)
    run = PagedRun(cfg, 3, B, 128)
    run.bb.set_option(vc.OPT_GRAPH, graph)
    run.bb.set_option(vc.OPT_FRAME, 1)     # has no effect on a paged step
    run.bb.set_taps(run.hid, run.lg)
    for t in range(frames):
        ro = run.step(t)
        check_step(run, ro)
    assert run.st.ctx_len.tolist() == [frames] * B and run.cache.lens.tolist() == [frames] * B
    assert int(run.st.status[0]) == 0 and int(run.cache.status[0]) == 0
    assert int((run.cache.refs > 0).sum()) == B * -(-frames // 16)


@pytest.mark.parametrize("pattern,wfmt,B", [("M*-", synth.FMT_BF16, 1), ("*-", synth.FMT_W4, 16), ("*M", synth.FMT_W8, 3)])
def test_nano_layers_match_the_oracle(cuda, pattern, wfmt, B):
    """the layers at the Nano widths, slots in another order than the rows"""
    cfg = nano_layer_cfg(pattern, wfmt, 128 if wfmt == synth.FMT_W8 else 64)
    run = PagedRun(cfg, 6, B, 64, page=64)
    for t in range(3):
        ro = run.step(t, slots=list(range(B))[::-1])
        hid = run.hid.cpu().numpy()
        for l in range(cfg.n_layers + 1):
            d = hid[l] - ro["hidden"][l]
            assert np.abs(d).max() <= TOL * np.sqrt(np.mean(np.square(ro["hidden"][l], dtype=np.float64))), (t, l)
    assert int(run.cache.status[0]) == 0


class PagedPrefillRun(PrefillRun):
    def __init__(self, cfg, seed, T, cap, page=32):
        super().__init__(cfg, seed, T, cap)
        columns = -(-cap // page)
        self.cache = self.bb.new_cache(columns + 3, page, columns)
        self.rows = self.st        # check_state reads k and v from rows that the test fills from the pages
        bb, cache = self.bb, self.cache
        bb.prefill = lambda x, slot, st: bb.prefill_paged(x, slot, st, cache)
        bb.step = lambda x, st, tt, tf: bb.step_paged(x, st, cache, tt, tf)

    def gather(self):
        for a in range(self.cfg.n_attn):
            n = int(self.cache.lens[0])
            p = self.cache.page_size
            for rows, pages in ((self.st.k, self.cache.k), (self.st.v, self.cache.v)):
                got = pages[a][self.cache.table[0][:-(-n // p)].long()].transpose(0, 1)   # [heads][columns][page][dim]
                rows[a, 0, :, :n] = got.reshape(got.shape[0], -1, got.shape[-1])[:, :n]


@pytest.mark.parametrize("wfmt", [synth.FMT_W8, synth.FMT_BF16])
@pytest.mark.parametrize("T", [1, 600])
def test_prefill_then_frames_match_the_oracle(cuda, wfmt, T):
    run = PagedPrefillRun(synth.tiny_config(wfmt=wfmt, head_fmt=wfmt), 7, T, T + 64)
    run.prefill()
    run.gather()
    run.check_state()
    assert run.steps(8) > 0
    assert int(run.cache.lens[0]) == T + 8


@pytest.mark.parametrize("wfmt", [synth.FMT_W4, synth.FMT_BF16])
def test_nano_attention_prefill_matches_the_oracle(cuda, wfmt):
    run = PagedPrefillRun(nano_layer_cfg("*", wfmt=wfmt), 9, 300, 364, page=64)
    run.prefill()
    run.gather()
    run.check_state()
    run.steps(2)


class WindowedLayer:
    """The attention layer l by its equations in 64 bits over a window with sinks, one session, and how far the step's
    roundings can take it.  Its operands are the path's own: u = bf16(fp32(r gamma)), weights bf16 or s (q - z), which
    a frame applies as they are (the scale multiplies a group's fp32 sum) and a prefill rounds to fp16.  The
    projections' fp32 sum of K terms is off by at most e = (K + 8) 2^-24 sum |u w| / rms.
      k, v: in the pages, one rounding to bf16: 2^-8 of the value, plus e
      q: stored in bf16 too; a value whose exact sum lies within e of a rounding boundary may have gone to the other
        neighbour, one step of at most 2^-7 of it; the flips of a head move a score by at most
        f = max over keys of scale sum 2^-7 |q_d k_d| over such d, every weight by a factor within exp(+-f), and so the
        quotient by at most (exp(2 f) - 1) sum w |v|
      o: the attention's own bound (paged_reference.tolerance, one rounding to bf16 included)
      what the layer adds: sum |w_o| times o's bound, (K + 8) 2^-24 sum |w_o o| for the sum, 2^-22 of the residual."""

    def __init__(self, om, l, window, sinks):
        self.cfg, self.window, self.sinks = om.cfg, window, sinks
        weights = [om.mats[(l, kind)].dequant() for kind in (synth.K_QKV, synth.K_O)]
        half = om.cfg.wfmt != synth.FMT_BF16
        self.weights = {"frame": weights, "prefill": [w.astype(np.float16).astype(float) if half else w for w in weights]}
        self.gamma = om.small[l]["norm"].astype(np.float32)

    def added(self, path, r, first, K, V, window=True):
        """(what the layer adds to the residual rows r [rows][d] at positions first.., its bound); K, V [positions][KV
        heads][dim]: what the pages hold up to the last row's position"""
        c = self.cfg
        Hq, Hk, Dh = c.attn_q_heads, c.attn_kv_heads, c.attn_head_dim
        w_qkv, w_o = self.weights[path]
        r = np.asarray(r, np.float32)
        u = mirror_layer.bf16(r * self.gamma)
        inv = 1.0 / np.sqrt(np.mean(r.astype(np.float64) ** 2, axis=-1, keepdims=True) + c.eps)
        exact = (u @ w_qkv.T) * inv
        slack = (u.shape[1] + 8) * 2.0 ** -24 * (np.abs(u) @ np.abs(w_qkv).T) * inv
        q = mirror_layer.bf16(exact)
        n_q, n_kv = Hq * Dh, Hk * Dh
        for got, at in ((K, n_q), (V, n_q + n_kv)):
            want, sl = exact[:, at:at + n_kv], slack[:, at:at + n_kv]
            assert (np.abs(got[first:].reshape(len(r), -1) - want) <= 2.0 ** -8 * (np.abs(want) + sl) + sl).all()
        flips = np.where(mirror_layer.bf16(exact + slack) != mirror_layer.bf16(exact - slack), 2.0 ** -7 * np.abs(q), 0.0)
        scale = default_scale(Dh)
        out, bound = np.empty((len(r), n_q)), np.empty((len(r), n_q))
        for i in range(len(r)):
            seen = seen_keys(first + i, len(K), self.window if window else 0, self.sinks)
            for h in range(Hq):
                j, d = h * Hk // Hq, slice(h * Dh, (h + 1) * Dh)
                o, absw, dots, abs_seen = attend_row(q[i, d], K[:, j], V[:, j], seen, scale)
                f = float((np.abs(K[seen, j]) @ flips[i, d]).max()) * scale
                out[i, d] = o
                bound[i, d] = tolerance(o, absw, dots, abs_seen, Dh, HALF_STEP["bf16"], FLOOR["bf16"]) + np.expm1(2 * f) * absw
        wo = np.abs(w_o).T
        add = out @ w_o.T
        return add, bound @ wo + (n_q + 8) * 2.0 ** -24 * (np.abs(out) @ wo) + 2.0 ** -22 * (np.abs(r) + np.abs(add))


def assert_added(hid, l, want, bound):
    got = hid[l + 1].astype(np.float64) - hid[l].astype(np.float64)
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


def assert_far(full, want, bound):
    assert (np.abs(full - want) / bound).max() > 5


def page_rows(cache, at):
    """(k, v) of session 0's positions at in the first layer, [positions][KV heads][dim]"""
    at = np.asarray(at)
    page = cache.table[0].cpu().numpy()[at // cache.page_size]
    assert (page >= 0).all()
    return [t[0, page, :, at % cache.page_size].double().cpu().numpy() for t in (cache.k, cache.v)]


@pytest.mark.parametrize("wfmt", [synth.FMT_W8, synth.FMT_BF16])
def test_frames_beyond_the_window(cuda, wfmt):
    """150 frames of one session through a window of 24 with 5 sinks: the pages in use stop growing"""
    cfg = synth.tiny_config(wfmt=wfmt, head_fmt=wfmt)
    window, sinks, page, frames = 24, 5, 16, 150
    run = PagedRun(cfg, 4, 1, 64, page=page, window=window, sinks=sinks, pages=4, columns=-(-frames // page))
    l = cfg.pattern.index("*")
    ref = WindowedLayer(run.om, l, window, sinks)
    K, V = np.empty((0, 2, 64)), np.empty((0, 2, 64))
    for t in range(frames):
        run.bb.step_paged(bits(synth.frame_inputs(cfg, 4, t, 1)), run.st, run.cache, run.tt, run.tf)
        hid = run.hid.cpu().numpy()
        k, v = page_rows(run.cache, [t])
        K, V = np.concatenate([K, k]), np.concatenate([V, v])
        want, bound = ref.added("frame", hid[l], t, K, V)
        assert_added(hid, l, want, bound)
        assert int(run.tt[0]) >= 0
    assert_far(ref.added("frame", hid[l], t, K, V, window=False)[0], want, bound)
    assert int((run.cache.refs > 0).sum()) <= 4 and int(run.cache.status[0]) == 0
    assert run.st.ctx_len.tolist() == [frames] == run.cache.lens.tolist()


@pytest.mark.parametrize("wfmt", [synth.FMT_W8, synth.FMT_BF16])
def test_prefill_beyond_the_window_then_frames(cuda, wfmt):
    import torch
    cfg = synth.tiny_config(wfmt=wfmt, head_fmt=wfmt)
    T, window, sinks, page = 201, 40, 3, 32
    run = PagedRun(cfg, 5, 1, 256, page=page, window=window, sinks=sinks, pages=8)
    l = cfg.pattern.index("*")
    ref = WindowedLayer(run.om, l, window, sinks)
    tap = torch.zeros((cfg.n_layers + 1, T, cfg.d_model), dtype=torch.float32, device="cuda")
    run.bb.set_prefill_taps(tap)
    run.bb.prefill_paged(bits(synth.prefill_inputs(cfg, 5, T)), 0, run.st, run.cache)
    run.bb.set_prefill_taps(None)
    hid = tap.cpu().numpy()
    K, V = page_rows(run.cache, range(T))
    want, bound = ref.added("prefill", hid[l], 0, K, V)
    assert_added(hid, l, want, bound)
    assert_far(ref.added("prefill", hid[l], 0, K, V, window=False)[0], want, bound)
    assert run.cache.lens.tolist() == [T] and int((run.cache.refs > 0).sum()) == 7
    for t in range(40):
        run.bb.step_paged(bits(synth.frame_inputs(cfg, 5, t, 1)), run.st, run.cache, run.tt, run.tf)
        hid = run.hid.cpu().numpy()
        k, v = page_rows(run.cache, [T + t])
        K, V = np.concatenate([K, k]), np.concatenate([V, v])
        assert_added(hid, l, *ref.added("frame", hid[l], T + t, K, V))
    # the first column holds the sinks; the columns behind the window went back
    assert (run.cache.table[0] >= 0).tolist() == [True] + 5 * [False] + [True, True]
    assert int(run.cache.status[0]) == 0


def test_a_row_without_room_is_skipped(cuda):
    """pages for one session's third page only: the other is skipped until it gets one"""
    cfg = synth.tiny_config()
    run = PagedRun(cfg, 8, 2, 64, pages=5)
    for t in range(32):
        run.step(t)
    before = run.st.ssm[:, 1].clone(), run.st.conv[:, 1].clone()
    run.step(32)
    assert int(run.cache.status[0]) == CAPACITY and int(run.st.status[0]) == 0
    assert int(run.tt[0]) >= 0 and run.tt.tolist()[1] == -1 and run.tf.tolist()[1] == -1
    assert run.st.ctx_len.tolist() == [33, 32] == run.cache.lens.tolist()
    assert bool((run.st.ssm[:, 1] == before[0]).all()) and bool((run.st.conv[:, 1] == before[1]).all())
    run.cache.resize(seqs=i32([0]), lens=i32([0]))       # session 0 ends; session 1 goes on
    run.step(33)
    assert run.tt.tolist()[1] >= 0 and run.cache.lens.tolist() == [1, 33]


def test_a_slot_named_twice_steps_once(cuda):
    cfg = synth.tiny_config()
    run = PagedRun(cfg, 8, 2, 64)
    run.bb.step_paged(bits(synth.frame_inputs(cfg, 8, 0, 2)), run.st, run.cache, run.tt, run.tf, slots=i32([1, 1]))
    assert run.tt.tolist()[0] >= 0 and run.tt.tolist()[1] == -1
    assert run.cache.lens.tolist() == [0, 1] == run.st.ctx_len.tolist() and int(run.cache.status[0]) == INVALID


def test_slots_out_of_range_are_skipped(cuda):
    cfg = synth.tiny_config()
    run, alone = PagedRun(cfg, 8, 3, 64), PagedRun(cfg, 8, 3, 64)
    for t in range(3):
        x = bits(synth.frame_inputs(cfg, 8, t, 3))
        run.bb.step_paged(x, run.st, run.cache, run.tt, run.tf, slots=i32([-1, 1, 1 << 30]))
        alone.bb.step_paged(x, alone.st, alone.cache, alone.tt, alone.tf, slots=i32([0, 1, 2]))
        assert run.tt.tolist()[0] == -1 == run.tt.tolist()[2] and run.tt.tolist()[1] >= 0
        a, b = run.hid[:, 1].double(), alone.hid[:, 1].double()
        assert float((a - b).abs().max()) <= TOL * float(b.square().mean().sqrt())
    assert run.cache.lens.tolist() == [0, 3, 0] == run.st.ctx_len.tolist() and int(run.cache.status[0]) == INVALID
    assert not bool(run.st.ssm[:, 0].any()) and not bool(run.st.ssm[:, 2].any())


def test_prefill_without_room_leaves_the_slot_empty(cuda):
    cfg = synth.tiny_config()
    run = PagedRun(cfg, 8, 2, 64, pages=3)
    x = bits(synth.prefill_inputs(cfg, 8, 60))
    run.bb.prefill_paged(x[:40], 0, run.st, run.cache)
    assert run.cache.lens.tolist() == [40, 0] and int(run.cache.status[0]) == 0
    run.bb.prefill_paged(x[:20], 1, run.st, run.cache)
    assert run.cache.lens.tolist() == [40, 0] == run.st.ctx_len.tolist() and int(run.cache.status[0]) == CAPACITY
    run.bb.prefill_paged(x[:48], 0, run.st, run.cache)   # over what the slot held
    assert run.cache.lens.tolist() == [48, 0] == run.st.ctx_len.tolist()
    run.bb.prefill_paged(x[:60], 0, run.st, run.cache)
    assert run.cache.lens.tolist() == [0, 0] == run.st.ctx_len.tolist() and int((run.cache.refs > 0).sum()) == 0


def test_forked_sessions_go_on_as_their_source(cuda):
    """an opening context shared by three sessions: the same inputs give the same frames, other inputs others, and
    the source goes on as if alone; the pages move in between"""
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    x = bits(synth.prefill_inputs(cfg, 2, 43))
    frames = synth.frame_inputs(cfg, 2, 0, 3)

    def opened(B):
        run = PagedRun(cfg, 2, B, 128, page=16, pages=40)
        run.bb.prefill_paged(x, 0, run.st, run.cache)
        return run

    alone, run = opened(1), opened(3)
    parts = vc.session_parts([run.st.ssm, run.st.conv, run.st.ctx_len])
    done = i32([0, 0])
    run.cache.fork(i32([0, 0]), i32([1, 2]), parts=parts, done=done)
    assert done.tolist() == [1, 1] and int((run.cache.refs == 3).sum()) == 2
    for t in range(20):
        if t == 7:
            run.cache.compact()
        same = np.repeat(frames[:1], 3, 0).copy()
        if t >= 10:
            same[2] = frames[2]
        run.step(t, x=same)
        alone.step(t, x=frames[:1])
        # split rows of the projections are summed in an order that varies: no equality bit for bit
        a, rms = run.hid.double(), float(run.hid[:, 0].double().square().mean().sqrt())
        assert float((a[:, 0] - alone.hid[:, 0]).abs().max()) <= TOL * rms
        assert float((a[:, 0] - a[:, 1]).abs().max()) <= TOL * rms
        assert (float((a[:, 0] - a[:, 2]).abs().max()) <= TOL * rms) == (t < 10)
    assert run.cache.lens.tolist() == [63] * 3 == run.st.ctx_len.tolist() and int(run.cache.status[0]) == 0


def test_fused_inputs(cuda):
    """the previous frame's tokens fused in: as the plain frame on the fused input"""
    import torch
    cfg = synth.tiny_config()
    gen = torch.Generator(device="cuda").manual_seed(3)
    emb = [torch.randn((v, cfg.d_model), generator=gen, device="cuda").bfloat16() for v in (cfg.vocab_text, cfg.vocab_func)]
    a, b = PagedRun(cfg, 2, 2, 64), PagedRun(cfg, 2, 2, 64)
    a.tt.fill_(-1)
    a.tf.fill_(-1)
    for t in range(5):
        x = bits(synth.frame_inputs(cfg, 2, t, 2))
        f = x.float()
        for toks, e in ((a.tt, emb[0]), (a.tf, emb[1])):
            f = f + torch.where(toks[:, None] >= 0, e[toks.clamp(min=0).long()].float(), torch.zeros_like(f))
        a.bb.step_paged(x, a.st, a.cache, a.tt, a.tf, emb=emb)
        b.bb.step_paged(f.bfloat16(), b.st, b.cache, b.tt, b.tf)
        assert torch.equal(a.hid[0], b.hid[0])
        assert float((a.hid - b.hid).abs().max()) <= TOL * float(b.hid.square().mean().sqrt())


def test_two_caches_take_turns(cuda):
    """one backbone over two caches and states: each call's graph belongs to its own"""
    import torch
    cfg = synth.tiny_config()
    one = PagedRun(cfg, 3, 2, 64)
    two = PagedRun(cfg, 3, 2, 64)
    cache, st = one.bb.new_cache(8, 16, 4, window=20, sinks=1), one.dm.new_state(2, 0)
    ref_cache = two.bb.new_cache(8, 16, 4, window=20, sinks=1)
    for t in range(30):
        x = bits(synth.frame_inputs(cfg, 3, t, 2))
        one.bb.step_paged(x, one.st, one.cache, one.tt, one.tf)
        one.bb.step_paged(x, st, cache, one.tt, one.tf)
        two.bb.step_paged(x, two.st, ref_cache, two.tt, two.tf)
    torch.cuda.synchronize()
    assert torch.equal(cache.table, ref_cache.table)
    assert one.cache.lens.tolist() == [30, 30] == cache.lens.tolist()
    assert float((one.hid - two.hid).abs().max()) <= TOL * float(two.hid.square().mean().sqrt())


def test_frames_in_a_callers_graph(cuda):
    """with direct launches a frame can be captured by the caller: every replay is the next frame"""
    import torch
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    one, two = PagedRun(cfg, 4, 2, 64, window=20, sinks=2), PagedRun(cfg, 4, 2, 64, window=20, sinks=2)
    one.bb.set_option(vc.OPT_GRAPH, 0)
    one.bb.set_taps(one.hid, one.lg)
    x = torch.zeros((2, cfg.d_model), dtype=torch.bfloat16, device="cuda")
    frame = lambda run: run.bb.step_paged(x, run.st, run.cache, run.tt, run.tf)  # noqa: E731
    x.copy_(bits(synth.frame_inputs(cfg, 4, 0, 2)))
    for run in (one, two):
        frame(run)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        frame(one)
    for t in range(1, 40):
        x.copy_(bits(synth.frame_inputs(cfg, 4, t, 2)))
        graph.replay()
        frame(two)
        assert float((one.hid - two.hid).abs().max()) <= TOL * float(two.hid.square().mean().sqrt())
    assert one.cache.lens.tolist() == [40, 40] == two.cache.lens.tolist() and torch.equal(one.cache.table, two.cache.table)
    assert int(one.cache.status[0]) == 0


def test_refusals(cuda):
    import torch
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    run = PagedRun(cfg, 1, 2, 64)
    x = bits(synth.frame_inputs(cfg, 1, 0, 2))
    shape = dict(layers=1, pages=8, page_size=16, kv_heads=2, head_dim=64, seqs=2, columns=4, q_heads=4)
    for bad in (dict(layers=2), dict(kv_heads=4), dict(head_dim=32), dict(q_heads=8), dict(seqs=3),
                dict(dtype=torch.float16)):
        cache = vc.PagedCache.empty(**{**shape, **bad})
        for call in (lambda: run.bb.step_paged(x, run.st, cache, run.tt, run.tf),
                     lambda: run.bb.prefill_paged(x, 0, run.st, cache)):
            with pytest.raises(vc.VcError) as e:
                call()
            assert e.value.code == vc.VC_ERR_INVALID_ARG
    small = vc.PagedCache.empty(**{**shape, "columns": 3})
    long = torch.zeros((65, cfg.d_model), dtype=torch.bfloat16, device="cuda")
    for rows, slot, cache, code in ((65, 0, run.cache, vc.VC_ERR_CAPACITY), (49, 0, small, vc.VC_ERR_CAPACITY),
                                    (0, 0, run.cache, vc.VC_ERR_INVALID_ARG), (4, 2, run.cache, vc.VC_ERR_INVALID_ARG),
                                    (4, -1, run.cache, vc.VC_ERR_INVALID_ARG)):
        with pytest.raises(vc.VcError) as e:
            run.bb.prefill_paged(long[:rows], slot, run.st, cache)
        assert e.value.code == code
    with pytest.raises(vc.VcError) as e:
        run.bb.step_paged(x[:0], run.st, run.cache, run.tt, run.tf)
    assert e.value.code == vc.VC_ERR_INVALID_ARG
    with pytest.raises(vc.VcError) as e:      # a table missing
        run.bb.step_paged(x, run.st, run.cache, run.tt, run.tf, emb=(None, x))
    assert e.value.code == vc.VC_ERR_INVALID_ARG
    assert int(run.cache.lens.sum()) == 0 and int(run.st.ctx_len.sum()) == 0
