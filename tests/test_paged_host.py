"""The paged KV cache without a GPU: the calls' refusals on the host (nothing is launched), the binding's
structures against the header, and the plain references' own pins."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import paged_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def vc():
    import attention_frame_decode_b200 as m
    return m


def kv(**kw):
    """a structure that passes the host checks; its pointers are never followed by them"""
    c = vc().VcPagedKv()
    for i, f in enumerate(("k", "v", "table", "len", "refs", "status", "workspace")):
        setattr(c, f, 0x10000 * (i + 1))
    c.layers, c.pages, c.page_size, c.kv_heads, c.head_dim, c.q_heads, c.f16 = 2, 64, 64, 8, 128, 40, 0
    c.seqs, c.columns, c.window, c.sinks = 16, 32, 1024, 4
    c.workspace_bytes = 1 << 40
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_SIZES = [dict(layers=0), dict(pages=0), dict(page_size=48), dict(page_size=8), dict(page_size=512), dict(kv_heads=0),
             dict(q_heads=12), dict(q_heads=0), dict(head_dim=96), dict(head_dim=512), dict(seqs=0), dict(columns=0),
             dict(window=-1), dict(sinks=-1), dict(columns=1 << 25), dict(pages=1 << 23), dict(seqs=1 << 27)]


@pytest.mark.parametrize("bad", BAD_SIZES, ids=str)
def test_sizes_outside_the_limits_have_no_workspace(bad):
    m = vc()
    c = kv(**bad)
    assert m.lib().vc_paged_workspace_bytes(ctypes.byref(c)) == 0
    assert m.lib().vc_paged_resize(ctypes.byref(c), 1, None, None, 1, None, None) == m.VC_ERR_INVALID_ARG


def test_workspace_grows_with_the_cache():
    m = vc()
    size = lambda **kw: m.lib().vc_paged_workspace_bytes(ctypes.byref(kv(**kw)))  # noqa: E731
    assert m.lib().vc_paged_workspace_bytes(None) == 0
    assert 0 < size() < size(pages=4096) and size() < size(seqs=4096)
    assert size() == size(k=None, workspace=None, workspace_bytes=0)   # pointers are not looked at


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=8), dict(table=None), dict(len=None), dict(refs=4), dict(status=None),
                                 dict(status=2), dict(workspace=None), dict(workspace=24), dict(workspace_bytes=1024)], ids=str)
def test_every_call_refuses_a_bad_cache(bad):
    m = vc()
    lib, c = m.lib(), ctypes.byref(kv(**bad))
    r = good_rows()
    assert lib.vc_paged_resize(c, 1, None, None, 1, None, None) == m.VC_ERR_INVALID_ARG
    assert lib.vc_paged_fork(c, 1, 16, 32, None, 0, None, None) == m.VC_ERR_INVALID_ARG
    assert lib.vc_paged_compact(c, None, None) == m.VC_ERR_INVALID_ARG
    assert lib.vc_paged_attend(c, 0, ctypes.byref(r), None) == m.VC_ERR_INVALID_ARG
    assert lib.vc_paged_attend(None, 0, ctypes.byref(r), None) == m.VC_ERR_INVALID_ARG


def good_rows(**kw):
    a = vc().VcAttnRows()
    a.q, a.k, a.v, a.out, a.pos = 0x1000, 0x2000, 0x3000, 0x4000, 0x5000
    a.q_stride, a.out_stride, a.k_stride, a.v_stride = 40 * 128, 40 * 128, 8 * 128, 8 * 128
    a.batch, a.rows = 4, 4
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(pos=None), dict(k=None), dict(v=None), dict(q=8),
                                 dict(out=8), dict(k=4), dict(pos=2), dict(seqs=1), dict(cu_rows=3), dict(batch=0),
                                 dict(batch=17, rows=17), dict(rows=0), dict(rows=5), dict(q_stride=40 * 128 - 8),
                                 dict(q_stride=40 * 128 + 4), dict(out_stride=8), dict(k_stride=8 * 128 - 8),
                                 dict(v_stride=8 * 128 + 1), dict(scale=float("nan")), dict(scale=float("inf")),
                                 dict(cu_rows=0x6000, rows=1 << 29)], ids=str)
def test_attend_refuses_bad_rows(bad):
    m = vc()
    assert m.lib().vc_paged_attend(ctypes.byref(kv()), 0, ctypes.byref(good_rows(**bad)), None) == m.VC_ERR_INVALID_ARG


@pytest.mark.parametrize("layer", [-1, 2])
def test_attend_refuses_a_layer_out_of_range(layer):
    m = vc()
    assert m.lib().vc_paged_attend(ctypes.byref(kv()), layer, ctypes.byref(good_rows()), None) == m.VC_ERR_INVALID_ARG


@pytest.mark.parametrize("n,seqs,lens,pos", [(0, None, None, None), (17, None, None, None), (1, 2, None, None),
                                             (1, None, 3, None), (1, None, None, 1)])
def test_resize_refuses_bad_arguments(n, seqs, lens, pos):
    m = vc()
    assert m.lib().vc_paged_resize(ctypes.byref(kv()), n, seqs, lens, 0, pos, None) == m.VC_ERR_INVALID_ARG


def test_fork_refuses_bad_arguments():
    m = vc()
    c = ctypes.byref(kv())

    def call(n=1, src=16, dst=32, part=None, n_parts=0):
        parts = (m.VcSessionPart * 1)()
        if part:
            for k, v in dict(dict(base=4096, bytes=64, stride=64, outer_stride=1024, outer=2), **part).items():
                setattr(parts[0], k, v)
        return m.lib().vc_paged_fork(c, n, src, dst, parts if part is not None else None, n_parts, None, None)

    for kw in (dict(n=0), dict(n=17), dict(src=None), dict(dst=None), dict(src=2), dict(n_parts=1), dict(n_parts=-1),
               dict(part={}, n_parts=9), dict(part=dict(base=None), n_parts=1), dict(part=dict(base=8), n_parts=1),
               dict(part=dict(bytes=0), n_parts=1), dict(part=dict(bytes=6), n_parts=1), dict(part=dict(stride=32), n_parts=1),
               dict(part=dict(outer=0), n_parts=1), dict(part=dict(outer_stride=1020), n_parts=1)):
        assert call(**kw) == m.VC_ERR_INVALID_ARG, kw


LAYOUT = r"""
#include <stddef.h>
#include <stdio.h>
#include "vc.h"
#define SZ(T) printf("%s %zu\n", #T, sizeof(T))
#define OFF(T, m) printf("%s.%s %zu\n", #T, #m, offsetof(T, m))
int main(void) {
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a host C compiler")
def test_binding_structs_match_the_header(tmp_path):
    m = vc()
    py = {"vc_paged_kv": m.VcPagedKv, "vc_session_part": m.VcSessionPart, "vc_attn_rows": m.VcAttnRows}
    lines = [f"SZ({n});" for n in py] + [f"OFF({n}, {f[0]});" for n, c in py.items() for f in c._fields_]
    src, exe = tmp_path / "layout.c", str(tmp_path / "layout")
    src.write_text(LAYOUT + "\n".join(lines) + "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I" + os.path.join(ROOT, "include"),
                    "-o", exe, str(src)], check=True, capture_output=True, timeout=300)
    for line in subprocess.run([exe], check=True, capture_output=True, text=True, timeout=60).stdout.splitlines():
        name, value = line.split()
        struct, _, member = name.partition(".")
        assert (getattr(py[struct], member).offset if member else ctypes.sizeof(py[struct])) == int(value), name


# ---- the references' own pins -------------------------------------------------------------------


def test_reference_attention_is_the_softmax():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=8), rng.normal(size=(5, 8)), rng.normal(size=(5, 8))
    out, *_ = ref.attend_row(q, k, v, np.array([True, False, True, True, False]), 0.5)
    w = np.exp(0.5 * k[[0, 2, 3]] @ q)
    np.testing.assert_allclose(out, (w / w.sum()) @ v[[0, 2, 3]], rtol=1e-12)
    assert list(np.nonzero(ref.seen_keys(7, 10, 3, 2))[0]) == [0, 1, 5, 6, 7]
    assert list(np.nonzero(ref.seen_keys(2, 10, 0, 0))[0]) == [0, 1, 2]


def test_reference_book_by_hand():
    b = ref.Book(pages=6, page=16, seqs=3, columns=4, window=16, sinks=1)
    assert b.resize([0, 1], [40, 16]) == [0, 0]
    assert b.table[0][:3] == [0, 1, 2] and b.table[1][:1] == [3] and b.refs == [1, 1, 1, 1, 0, 0]
    assert b.fork([0, 0], [2, 2]) == [1, 0] and b.status == ref.INVALID        # the same session twice
    assert b.table[2][:3] == [0, 1, 4] and b.refs == [2, 2, 1, 1, 1, 0] and b.copies == [(2, 4, 8)]
    # position 48 opens a column; a query from 40 on sees 25.. and the sink's page: column 1 ends at 31, kept
    assert b.resize([0], [49]) == [40] and b.table[0] == [0, 1, 2, 5]
    # from 49 on a query sees 34..: column 1 (16..31) goes back for session 0, session 2 still has it
    assert b.resize([0], [50]) == [49] and b.table[0] == [0, -1, 2, 5] and b.refs[1] == 1
    assert b.resize([1], [33]) == [-1] and b.status == ref.INVALID | ref.CAPACITY
    assert b.resize([0], [20]) == [-1]                                         # inside a page given up
    assert b.resize([1], [0]) == [0] and b.compact() == (5, [(5, 3)])


def test_paged_steps_refuse_a_missing_backbone():
    m = vc()
    lib, c, st, emb = m.lib(), kv(), m.VcState(), m.VcTokenEmbeddings()
    for e in (None, ctypes.byref(emb)):
        assert lib.vc_step_paged(None, 16, e, 1, None, ctypes.byref(st), ctypes.byref(c), 16, 16, None) == m.VC_ERR_INVALID_ARG
    assert lib.vc_prefill_paged(None, 16, 1, 0, ctypes.byref(st), ctypes.byref(c), None) == m.VC_ERR_INVALID_ARG
