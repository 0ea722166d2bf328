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
