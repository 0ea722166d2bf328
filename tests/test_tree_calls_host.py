"""Draft-tree calls on the host: workspace sizes, and refusals before anything reaches a GPU."""

import ctypes as C
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from mtp_speculative_draft_gb300 import build, _lib
    build.build()
    return _lib.load()


def test_workspace_of_heads_that_do_not_group(lib):
    """Fewer query heads than KV heads, or a remainder: no size, and no arithmetic on zero tiles."""
    code = ("import ctypes as C; from mtp_speculative_draft_gb300 import _lib; lib = _lib.load()\n"
            "for nh, nkv in ((1, 2), (3, 4), (6, 4), (63, 64)):\n"
            "    g = _lib.AttnGeom(nh, nkv, 64, 64, 64, 0, 0, 1e-6, 0.0)\n"
            "    assert lib.attn_tree_sink_workspace_bytes(C.byref(g), 1, 100) == 0\n")
    assert subprocess.run([sys.executable, "-c", code], cwd=ROOT).returncode == 0


@pytest.mark.parametrize("nh,nkv,dqk,dv,window", [(40, 8, 128, 128, 0), (16, 2, 256, 256, 0), (4, 2, 64, 64, 0),
                                                  (32, 8, 192, 128, 128), (64, 1, 32, 256, 0), (7, 1, 96, 32, 3000)])
def test_workspace_of_the_largest_call_does_for_all(lib, nh, nkv, dqk, dv, window):
    """The size grows with the nodes and with the cached keys."""
    from mtp_speculative_draft_gb300 import _lib
    g = _lib.AttnGeom(nh, nkv, dqk, dv, dqk, window, 0, 1e-6, 0.0)
    lengths = list(range(0, 200, 3)) + list(range(1100, 1400)) + [4096, 4097, 8191, 32767, 32768]
    size = [[lib.attn_tree_sink_workspace_bytes(C.byref(g), n, L) for L in lengths] for n in range(1, 65)]
    for n, row in enumerate(size):
        assert all(a <= b for a, b in zip(row, row[1:]))
        assert n == 0 or all(a <= b for a, b in zip(size[n - 1], row))


def test_misaligned_workspaces_are_refused(lib):
    """The error word at the workspace's start takes an atomic: 4 bytes off, or 1, is refused."""
    from mtp_speculative_draft_gb300 import _lib
    P = C.c_void_p(0x100000)
    ax = _lib.RopeAxes(0x1000, 0x2000, 1, (C.c_int32 * 4)(64, 0, 0, 0), 0, 8, 100)
    rows = (_lib.HeadRows * 1)(_lib.HeadRows(0x10000, 0x20000, None, 1024, 1024, 128, 128, 8))
    caches = _lib.KvCaches((C.c_void_p * 1)(0x1000), (C.c_void_p * 1)(0x2000), 1, 2, 64, 64, 64)
    for ws in (0x100001, 0x100004, 0x100008):
        ws = C.c_void_p(ws)
        assert lib.mtp_tree_plan(P, 4, P, P, ws, 1024, None) == 4
        assert lib.mtp_token_counts(P, 10, P, 3, 0, ws, 1024, None) == 4
        assert lib.kv_tree_commit(C.byref(caches), P, 4, 0, ws, 1024, None) == 4
        assert lib.rope_axes_rows(C.byref(ax), rows, 1, 4, 128, 1e-6, ws, 1024, None) == 4


def test_a_call_that_makes_its_workspace_makes_it_on_its_stream(monkeypatch):
    """The buffer comes from the pool of the stream that uses it: another stream's pool would hand out memory that
    stream may still use, and take it back while this one does."""
    import torch
    from mtp_speculative_draft_gb300 import api
    current, made = [None], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *exc):
            current.pop()

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(current[-1]))
    monkeypatch.setattr(api, "mtp_workspace_init", lambda ws, stream=None: None)
    side = object()
    api.workspace(5000, stream=side)
    api.workspace(5000)
    assert made == [side, None]
