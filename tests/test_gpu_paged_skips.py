"""Batches of the paged cache's prompts in which most sessions have no position: what is handed out then has no key
blocks, piece after piece, between sessions that do."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_paged_edges import Sessions  # noqa: E402


@pytest.mark.parametrize("heads", [(8, 8, 64), (8, 8, 128)], ids=str)
@pytest.mark.parametrize("sessions", [400, 700])
def test_long_runs_of_skipped_sessions(heads, sessions):
    """twenty or more skipped pieces one behind another for every CTA: behind the others (tiles in order of their length,
    up to 512), or between sessions with rows; call after call"""
    live = [0, 90, 91, 300, sessions - 1]
    rows = [7] * sessions
    for i, n in zip(live, (260, 1, 40, 129, 33)):
        rows[i] = n
    ctx = [(31 * i) % 170 for i in range(sessions)]
    s = Sessions(heads, 16, "bf16", 90, 3, ctx, rows, seed=21)
    pos = [c if i in live else -1 for i, c in enumerate(ctx)]
    first = None
    for _ in range(8):
        out = s.run(pos=pos)
        assert first is None or torch.equal(out, first)
        first = out
    assert int(s.cache.status) == 0
    skipped = torch.ones(out.shape[0], dtype=torch.bool, device="cuda")
    for i in live:
        skipped[int(s.starts[i]):int(s.starts[i + 1])] = False
    assert torch.equal(out[skipped], torch.full_like(out[skipped], 7.0))
    r = np.random.default_rng(3)
    s.check(out, {(i, int(x)) for i in live for x in (0, rows[i] - 1, r.integers(rows[i]))})


@pytest.mark.parametrize("sessions", [30, 600])
def test_nobody_has_a_position(sessions):
    s = Sessions((8, 8, 64), 16, "bf16", 90, 3, [20] * sessions, [9] * sessions, seed=22)
    before = s.k.clone()
    for _ in range(3):
        out = s.run(pos=[-1] * sessions)
        assert torch.equal(out, torch.full_like(out, 7.0)) and torch.equal(s.k, before) and int(s.cache.status) == 0
