"""Infinities and NaN among the values that a row of the paged cache's attention sees.  Every seen key has a weight above
0, however small: a dimension whose seen values hold infinities of one sign is that infinity, one that holds both or NaN
is NaN, and the others are held to their bound."""
import numpy as np
import pytest

import paged_reference as ref

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_paged import Setup  # noqa: E402

INF, NAN = float("inf"), float("nan")


def place(s, i, p, j, dim, value):
    """value in dimension dim of position p of session i, KV head j: in its page, or among the new rows"""
    if p < s.ctx[i]:
        s.v[0, s.table[s.seqs[i], p // s.page].long(), j, p % s.page, dim] = value
    else:
        s.parts()[2][int(s.starts[i]) + p - s.ctx[i], j, dim] = value


def check(s, out, rows, scale=None):
    """rows: (session, row) pairs"""
    scale = ref.default_scale(s.d) if scale is None else scale
    got = out.float().cpu().numpy()
    q = s.parts()[0].float().cpu().numpy()
    kinds = set()
    for i, nth in rows:
        c, n = s.ctx[i], s.rows[i]
        keys, values = s.history(i), s.history(i, v=True)
        seen = ref.seen_keys(c + nth, c + n, s.window, s.sinks)
        for h in range(s.hq):
            j = h * s.hk // s.hq
            v = values[seen, j]
            up, down, nan = (v == INF).any(0), (v == -INF).any(0), np.isnan(v).any(0)
            o, a, z, av = ref.attend_row(q[s.starts[i] + nth, h], keys[:, j], np.where(np.isfinite(values[:, j]), values[:, j], 0),
                                         seen, scale)
            want = np.where(nan | (up & down), NAN, np.where(up, INF, np.where(down, -INF, o)))
            y = got[s.starts[i] + nth, h]
            odd = ~np.isfinite(want)
            kinds |= {str(x) for x in want[odd]}
            assert np.array_equal(y[odd], want[odd], equal_nan=True), (i, nth, h, y[odd], want[odd])
            tol = ref.tolerance(o, a, z, av, s.d, ref.HALF_STEP[s.dtype], ref.FLOOR[s.dtype])
            assert np.all(np.abs(y - o)[~odd] <= tol[~odd]), (i, nth, h)
    assert kinds == {"inf", "-inf", "nan"} and int(s.cache.status) == 0


def spread(s):
    """values that are not finite all over what session 0's rows see, sinks, window's edge, old pages, the newest row: one
    sign in six dimensions, both in another, NaN in another"""
    n = s.ctx[0] + s.rows[0]
    first = 0 if not s.window else max(s.ctx[0] - s.window + 1, 0)
    at = [0, first, first + (n - first) // 3, (first + n) // 2, n - 20, s.ctx[0]]
    dims = [0, s.d // 2 + 1, s.d - 1, s.d // 4 + 2, 5, s.d // 2 - 2]
    for k, (p, dim) in enumerate(zip(at, dims)):
        place(s, 0, p, 0, dim, INF if k % 2 else -INF)
    place(s, 0, at[2], 0, s.d // 2 + 4, INF)
    place(s, 0, at[4], 0, s.d // 2 + 4, -INF)
    place(s, 0, at[3], 0, s.d - 9, NAN)


FRAMES = [((4, 2, 64), 32, 0, 0, 700), ((40, 8, 128), 64, 300, 5, 2100), ((8, 2, 32), 16, 100, 30, 517),
          ((8, 4, 256), 32, 0, 0, 900), ((16, 1, 256), 64, 0, 0, 3000), ((12, 1, 64), 16, 700, 3, 9000),
          ((5, 1, 128), 64, 0, 0, 30011), ((8, 8, 64), 64, 0, 0, 260)]


@pytest.mark.parametrize("scale", [0.0, 30.0])        # 30: most weights are 0 in 32 bits
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,page,window,sinks,ctx", FRAMES, ids=str)
def test_frames(heads, page, window, sinks, ctx, dtype, scale):
    s = Setup(heads, page, dtype, window, sinks, [ctx, 40], [1, 1], seed=31)
    spread(s)
    check(s, s.run(single=True, scale=scale), [(0, 0), (1, 0)], scale or None)


def test_frames_of_one_chunk_and_of_many_sessions():
    """(session, KV head)s that a warp has alone: nothing is joined"""
    s = Setup((8, 2, 64), 16, "bf16", 60, 2, [90] + [(13 * i) % 80 for i in range(600)], [1] * 601, seed=32)
    spread(s)
    check(s, s.run(single=True), [(0, 0), (1, 0), (600, 0)])


def test_frames_of_more_heads_than_the_frames_form_takes():
    for dtype, scale in (("bf16", 0.0), ("fp16", 0.0), ("fp16", 30.0)):
        s = Setup((34, 2, 64), 64, dtype, 129, 5, [800, 40], [1, 1], seed=34)
        spread(s)
        check(s, s.run(single=True, scale=scale), [(0, 0), (1, 0)], scale or None)


PROMPTS = [((4, 2, 64), 32, 0, 0, 500, 90), ((40, 8, 128), 64, 120, 4, 300, 150), ((8, 2, 32), 16, 100, 30, 300, 60),
           ((8, 4, 256), 32, 0, 0, 400, 70), ((8, 2, 64), 64, 0, 0, 12000, 5), ((8, 2, 128), 64, 0, 0, 12000, 5),
           ((8, 2, 32), 64, 0, 0, 12000, 5), ((8, 1, 256), 64, 0, 0, 12000, 5), ((8, 2, 64), 16, 0, 0, 1000, 3),
           ((8, 2, 128), 32, 0, 0, 2000, 1), ((2, 2, 64), 32, 0, 0, 0, 600), ((300, 1, 64), 32, 0, 0, 200, 3)]


@pytest.mark.parametrize("scale", [0.0, 30.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,page,window,sinks,ctx,rows", PROMPTS, ids=str)
def test_prompts(heads, page, window, sinks, ctx, rows, dtype, scale):
    """blocks that all rows see, blocks at the edges, ranges of keys joined at the end or by a launch of their own"""
    s = Setup(heads, page, dtype, window, sinks, [ctx, 40], [rows, 33], seed=35)
    spread(s)
    out = s.run(scale=scale)
    check(s, out, [(0, r) for r in sorted({0, rows // 3, rows // 2, rows - 1})] + [(1, 0), (1, 32)], scale or None)


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 2, 128), (8, 2, 32)])
def test_a_key_that_is_not_a_number_spoils_its_heads_alone(heads, single):
    s = Setup(heads, 32, "bf16", 0, 0, [3000, 50], [1, 1], seed=33)
    s.k[0, s.table[0, 40].long(), 0, 3, 5] = NAN
    place(s, 0, 100, 0, 1, INF)
    out = s.run(single=single)
    group = s.hq // s.hk
    assert torch.isnan(out[0, :group]).all() and torch.isfinite(out[0, group:]).all() and torch.isfinite(out[1]).all()
