"""Sessions of a backbone over a paged cache that end, start again, or lose their pages: the recurrent state follows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import synth  # noqa: E402
from paged_reference import CAPACITY, INVALID  # noqa: E402
from test_gpu_paged_backbone import TOL, PagedRun, bits, i32  # noqa: E402


def same_row(a, b, i, j):
    """row i of a's frame and row j of b's, over all layers (split rows of the projections are summed in varying order)"""
    x, y = a.hid[:, i].double(), b.hid[:, j].double()
    return float((x - y).abs().max()) <= TOL * float(y.square().mean().sqrt())


@pytest.mark.parametrize("graph", [0, 1])
@pytest.mark.parametrize("slots", [None, [2, 0, 1]])
def test_an_ended_session_starts_anew(cuda, slots, graph):
    """session of row 1 ends after 21 frames; its next frames are a fresh session's, and the others go on"""
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    run, fresh, on = PagedRun(cfg, 8, 3, 64, taps=False), PagedRun(cfg, 8, 3, 64, taps=False), PagedRun(cfg, 8, 3, 64, taps=False)
    for r in (run, fresh, on):
        r.bb.set_option(vc.OPT_GRAPH, graph)
        r.hid = torch.zeros((cfg.n_layers + 1, 3, cfg.d_model), device="cuda")
        r.bb.set_taps(r.hid)
    ended = (slots or [0, 1, 2])[1]
    sl = None if slots is None else i32(slots)
    step = lambda r, t: r.bb.step_paged(bits(synth.frame_inputs(cfg, 8, t, 3)), r.st, r.cache, r.tt, r.tf, slots=sl)  # noqa: E731
    for t in range(21):
        step(run, t)
        step(on, t)
    run.cache.resize(seqs=i32([ended]), lens=i32([0]))
    for t in range(21, 30):
        step(run, t)
        step(fresh, t)
        step(on, t)
        assert same_row(run, fresh, 1, 1) and same_row(run, on, 0, 0) and same_row(run, on, 2, 2)
        assert not same_row(run, on, 1, 1)
        want = [30 if s != ended else t - 20 for s in range(3)] if t == 29 else None
        assert want is None or run.cache.lens.tolist() == want == run.st.ctx_len.tolist()
    assert torch.equal(run.cache.status, i32([0])) and torch.equal(run.st.status, i32([0]))


def test_a_session_ended_twice_and_one_that_never_began(cuda):
    cfg = synth.tiny_config()
    run, fresh = PagedRun(cfg, 8, 2, 64), PagedRun(cfg, 8, 2, 64)
    x = bits(synth.prefill_inputs(cfg, 8, 40))
    run.bb.prefill_paged(x, 1, run.st, run.cache)
    for _ in range(2):
        run.cache.resize(seqs=i32([1]), lens=i32([0]))
        for r in (run, fresh):
            r.bb.step_paged(bits(synth.frame_inputs(cfg, 8, 0, 2)), r.st, r.cache, r.tt, r.tf)
        assert same_row(run, fresh, 1, 1) and run.st.ctx_len.tolist() == run.cache.lens.tolist()
        fresh.cache.resize(seqs=i32([1]), lens=i32([0]))


def test_a_first_frame_keeps_a_state_that_was_put_there(cuda):
    """ctx_len 0 and length 0: the session's state is the caller's, as in a step over rows"""
    cfg = synth.tiny_config()
    run, rows = PagedRun(cfg, 8, 1, 64), PagedRun(cfg, 8, 1, 64)
    rows.st = rows.dm.new_state(1, 64)
    for r in (run, rows):
        r.st.ssm.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
        r.st.conv.normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    x = bits(synth.frame_inputs(cfg, 8, 0, 1))
    run.bb.step_paged(x, run.st, run.cache, run.tt, run.tf)
    rows.bb.step(x, rows.st, rows.tt, rows.tf)
    assert same_row(run, rows, 0, 0)


@pytest.mark.parametrize("graph", [0, 1])
def test_a_state_of_another_position_is_not_stepped(cuda, graph):
    """a session cut back in the cache alone, one forked without its parts, one whose count was changed: each is skipped
    and stays as it is, the last goes on; with the state of their position they go on too"""
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    run, alone = PagedRun(cfg, 8, 4, 64), PagedRun(cfg, 8, 4, 64)
    run.bb.set_option(vc.OPT_GRAPH, graph)
    run.bb.set_taps(run.hid, run.lg)
    step = lambda r, t: r.bb.step_paged(bits(synth.frame_inputs(cfg, 8, t, 4)), r.st, r.cache, r.tt, r.tf)  # noqa: E731
    for t in range(10):
        step(run, t)
        step(alone, t)
    saved = [x.clone() for x in (run.st.ssm, run.st.conv)]
    for t in range(10, 20):
        step(run, t)
        step(alone, t)
    run.cache.resize(seqs=i32([0]), lens=i32([10]))
    run.st.ctx_len[1] = 3
    run.cache.resize(seqs=i32([2]), lens=i32([0]))
    run.cache.fork(i32([3]), i32([2]))                      # pages alone
    run.st.ctx_len[2] = 0
    keep = [x.clone() for x in (run.st.ssm[:, :3], run.st.conv[:, :3], run.st.ctx_len[:3], run.cache.lens[:3], run.cache.table[:3])]
    step(run, 20)
    step(alone, 20)
    assert run.tt.tolist()[:3] == [-1] * 3 == run.tf.tolist()[:3] and int(run.tt[3]) >= 0
    assert same_row(run, alone, 3, 3) and int(run.cache.status[0]) == INVALID and int(run.st.status[0]) == 0
    for a, b in zip(keep, (run.st.ssm[:, :3], run.st.conv[:, :3], run.st.ctx_len[:3], run.cache.lens[:3], run.cache.table[:3])):
        assert torch.equal(a, b)
    assert run.cache.lens.tolist() == [10, 20, 20, 21]
    # the state of the position that session 0 was cut back to
    run.st.ssm[:, 0], run.st.conv[:, 0] = saved[0][:, 0], saved[1][:, 0]
    run.st.ctx_len[0] = 10
    run.st.ctx_len[1] = 20
    for t in range(10, 14):
        step(run, t)
        assert int(run.tt[0]) >= 0 and int(run.tt[1]) >= 0
    assert run.cache.lens.tolist()[:2] == [14, 24] == run.st.ctx_len.tolist()[:2]


def test_a_session_cut_back_with_its_state_repeats_its_frames(cuda):
    cfg = synth.tiny_config()
    run = PagedRun(cfg, 8, 1, 64)
    for t in range(12):
        run.bb.step_paged(bits(synth.frame_inputs(cfg, 8, t, 1)), run.st, run.cache, run.tt, run.tf)
        if t == 6:
            saved = run.st.ssm.clone(), run.st.conv.clone()
        if t == 7:
            hid = run.hid.clone()
    run.cache.resize(lens=i32([7]))
    run.st.ssm.copy_(saved[0]), run.st.conv.copy_(saved[1])
    run.st.ctx_len.fill_(7)
    run.bb.step_paged(bits(synth.frame_inputs(cfg, 8, 7, 1)), run.st, run.cache, run.tt, run.tf)
    assert float((run.hid - hid).abs().max()) <= TOL * float(hid.square().mean().sqrt())


def test_a_slot_whose_prefill_had_no_room_is_a_fresh_one(cuda):
    """a used slot, then one that was never used: after a prefill without room their frames are a fresh session's"""
    cfg = synth.tiny_config()
    run, fresh = PagedRun(cfg, 8, 3, 64, pages=4), PagedRun(cfg, 8, 3, 64)
    x = bits(synth.prefill_inputs(cfg, 8, 64))
    run.bb.prefill_paged(x[:20], 0, run.st, run.cache)
    run.bb.prefill_paged(x[:16], 1, run.st, run.cache)
    other = [t[:, 1].clone() for t in (run.st.ssm, run.st.conv)]
    for slot in (0, 2):
        run.bb.prefill_paged(x[:60], slot, run.st, run.cache)
        assert int(run.cache.status[0]) == CAPACITY
        assert run.cache.lens.tolist() == [0, 16, 0] == run.st.ctx_len.tolist()
        assert not bool(run.st.ssm[:, slot].any()) and not bool(run.st.conv[:, slot].any())
        assert all(torch.equal(t[:, 1], o) for t, o in zip((run.st.ssm, run.st.conv), other))
    for t in range(3):
        for r in (run, fresh):
            r.bb.step_paged(bits(synth.frame_inputs(cfg, 8, t, 3)), r.st, r.cache, r.tt, r.tf)
        assert same_row(run, fresh, 0, 0) and same_row(run, fresh, 2, 2)
    assert run.st.ctx_len.tolist() == [3, 19, 3] == run.cache.lens.tolist()


def test_a_session_at_its_tables_end(cuda):
    """a windowed session has columns * page_size frames over its life, however few pages it holds: the next one is
    refused and changes nothing, others go on, and ended it starts anew"""
    cfg = synth.tiny_config()
    run = PagedRun(cfg, 8, 2, 64, page=16, window=20, sinks=3, pages=8, columns=5)
    run.bb.prefill_paged(bits(synth.prefill_inputs(cfg, 8, 60)), 0, run.st, run.cache)
    step = lambda t: run.bb.step_paged(bits(synth.frame_inputs(cfg, 8, t, 2)), run.st, run.cache, run.tt, run.tf)  # noqa: E731
    for t in range(20):
        step(t)
    assert run.cache.lens.tolist() == [80, 20] == run.st.ctx_len.tolist() and int(run.cache.status[0]) == 0
    step(20)                                                # (its window gives a page back all the same)
    assert run.tt.tolist()[0] == -1 == run.tf.tolist()[0] and int(run.tt[1]) >= 0
    keep = [x.clone() for x in (run.st.ssm[:, 0], run.st.conv[:, 0], run.cache.table[0])]
    held = (run.cache.table[0] >= 0).tolist()
    for t in range(21, 24):
        step(t)
        assert run.tt.tolist()[0] == -1 == run.tf.tolist()[0] and int(run.tt[1]) >= 0
    assert run.cache.lens.tolist() == [80, 24] == run.st.ctx_len.tolist()
    assert int(run.cache.status[0]) == CAPACITY and int(run.st.status[0]) == 0
    assert held == [True, False, False, True, True]
    for a, b in zip(keep, (run.st.ssm[:, 0], run.st.conv[:, 0], run.cache.table[0])):
        assert torch.equal(a, b)
    run.cache.resize(seqs=i32([0]), lens=i32([0]))
    step(24)
    assert int(run.tt[0]) >= 0 and run.cache.lens.tolist() == [1, 25] == run.st.ctx_len.tolist()


@pytest.mark.parametrize("graph", [0, 1])
def test_without_programmatic_launches(cuda, graph):
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    run, other = PagedRun(cfg, 5, 2, 96, window=30, sinks=2), PagedRun(cfg, 5, 2, 96, window=30, sinks=2)
    run.bb.set_option(vc.OPT_PDL, 0)
    run.bb.set_option(vc.OPT_GRAPH, graph)
    run.bb.set_taps(run.hid, run.lg)
    for r in (run, other):
        r.bb.prefill_paged(bits(synth.prefill_inputs(cfg, 5, 50)), 1, r.st, r.cache)
    for t in range(20):
        for r in (run, other):
            r.bb.step_paged(bits(synth.frame_inputs(cfg, 5, t, 2)), r.st, r.cache, r.tt, r.tf)
        assert same_row(run, other, 0, 0) and same_row(run, other, 1, 1)
    assert run.cache.lens.tolist() == [20, 70] and int(run.cache.status[0]) == 0


def test_a_smaller_pool_after_compact(cuda):
    """the first pages of every layer, refs cut to them, the same table and lengths: sessions go on over it"""
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    run, whole = PagedRun(cfg, 8, 3, 64, pages=40), PagedRun(cfg, 8, 3, 64, pages=40)
    for r in (run, whole):
        for slot, n in enumerate((40, 21, 33)):
            r.bb.prefill_paged(bits(synth.prefill_inputs(cfg, 8, n)), slot, r.st, r.cache)
        r.cache.resize(seqs=i32([0]), lens=i32([0]))
    live = i32([0])
    run.cache.compact(live=live)
    n = int(live) + 3
    c = run.cache
    run.cache = vc.PagedCache(c.k[:, :n].contiguous(), c.v[:, :n].contiguous(), c.table, c.lens, c.refs[:n].contiguous(),
                              q_heads=c.q_heads, window=c.window, sinks=c.sinks)
    for t in range(15):
        for r in (run, whole):
            r.bb.step_paged(bits(synth.frame_inputs(cfg, 8, t, 3)), r.st, r.cache, r.tt, r.tf)
        assert all(same_row(run, whole, i, i) for i in range(3))
    assert run.cache.lens.tolist() == [15, 36, 48] == run.st.ctx_len.tolist() and int(run.cache.status[0]) == 0
    assert int((run.cache.refs > 0).sum()) == 1 + 3 + 3


def test_a_session_whose_fork_found_no_page_starts_anew(cuda):
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    run, fresh = PagedRun(cfg, 8, 3, 64, pages=4), PagedRun(cfg, 8, 3, 64)
    x = bits(synth.prefill_inputs(cfg, 8, 40))
    run.bb.prefill_paged(x[:40], 0, run.st, run.cache)
    run.bb.prefill_paged(x[:9], 1, run.st, run.cache)
    parts = vc.session_parts([run.st.ssm, run.st.conv, run.st.ctx_len])
    done = i32([7, 7])
    run.cache.fork(i32([0, 0]), i32([1, 2]), parts=parts, done=done)      # one page is free once session 1's went back
    assert done.tolist() == [1, 0] and run.cache.lens.tolist() == [40, 40, 0] and int(run.cache.status[0]) == CAPACITY
    run.st.ctx_len[2] = 5                                                   # as if it had held frames
    run.st.ssm[:, 2] = 1.0
    run.cache.resize(seqs=i32([0, 1]), lens=i32([0, 0]))                    # four pages are free
    for t in range(3):
        for r in (run, fresh):
            r.bb.step_paged(bits(synth.frame_inputs(cfg, 8, t, 3)), r.st, r.cache, r.tt, r.tf)
        assert all(same_row(run, fresh, i, i) for i in range(3))
    assert run.cache.lens.tolist() == [3, 3, 3] == run.st.ctx_len.tolist()


@pytest.mark.parametrize("graph", [0, 1])
def test_every_session_ends_at_once(cuda, graph):
    """all sixteen rows start anew in one step, while slots that the step does not name keep their state"""
    import attention_frame_decode_b200 as vc
    cfg = synth.tiny_config()
    run, fresh = PagedRun(cfg, 8, 16, 64, pages=40), PagedRun(cfg, 8, 16, 64, pages=40)
    for r in (run, fresh):
        r.bb.set_option(vc.OPT_GRAPH, graph)
        r.bb.set_taps(r.hid, r.lg)
    step = lambda r, t, B=16: r.bb.step_paged(bits(synth.frame_inputs(cfg, 8, t, 16))[:B], r.st, r.cache, r.tt[:B], r.tf[:B])  # noqa: E731
    for t in range(5):
        step(run, t)
    run.cache.resize(lens=torch.zeros(16, dtype=torch.int32, device="cuda"))
    keep = [run.st.ssm[:, 12:].clone(), run.st.conv[:, 12:].clone(), run.st.ctx_len[12:].clone()]
    for r in (run, fresh):
        r.bb.set_taps(None, None)
        step(r, 0, 12)
        r.bb.set_taps(r.hid, r.lg)
    assert all(torch.equal(a, b[:, 12:] if b.dim() > 1 else b[12:]) for a, b in zip(keep, (run.st.ssm, run.st.conv, run.st.ctx_len)))
    for t in range(1, 4):
        for r in (run, fresh):
            step(r, t)
        assert all(same_row(run, fresh, i, i) for i in range(16))
    assert run.cache.lens.tolist() == [4] * 12 + [3] * 4 == run.st.ctx_len.tolist()
    assert fresh.st.ctx_len.tolist() == [4] * 12 + [3] * 4
