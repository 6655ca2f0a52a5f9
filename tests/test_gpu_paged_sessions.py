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
