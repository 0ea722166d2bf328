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
    monkeypatch.setattr(torch.cuda, "Stream", type("Stream", (), {}))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    side, handle = torch.cuda.Stream(), type("Handle", (), dict(cuda_stream=7))()  # any object with a cudaStream_t
    api.workspace(5000, stream=side)
    api.workspace(5000)
    api.workspace(5000, stream=handle)
    assert made == [side, None, ("external", 7)]


class _Tensor:
    """What the wrappers look at, of a tensor on a device that this machine need not have."""

    def __init__(self, device, dtype, *shape, stride=None):
        import math
        self.device, self.dtype, self.shape, self.is_cuda = device, dtype, shape, True
        self._stride = stride or tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))

    get_device = lambda self: self.device  # noqa: E731
    is_contiguous = lambda self: True  # noqa: E731
    data_ptr = lambda self: 0x100000  # noqa: E731
    dim = lambda self: len(self.shape)  # noqa: E731

    def numel(self):
        import math
        return math.prod(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]


class _Lib:
    """Counts what gets through to the library."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Workspaces and descriptors made on device 0, the current device is 1."""
    import torch
    from mtp_speculative_draft_gb300 import _lib, tree as W
    i32, i64, f32, u8 = torch.int32, torch.int64, torch.float32, torch.uint8
    current, lib = [0], _Lib()
    monkeypatch.setattr(W, "_device", lambda: current[0])
    monkeypatch.setattr(W, "_on", lambda stream, device: None)
    monkeypatch.setattr(_lib, "load", lambda: lib)

    def make(d):
        ax = W.rope_axes((32,), _Tensor(d, i32, 1, 3), _Tensor(d, f32, 10, 32, 2))
        return dict(ax=ax, tree=W.draft_tree(_Tensor(d, i64, 3), _Tensor(d, i32, 3), ax), ws=_Tensor(d, u8, 4096),
                    rules=W.logit_rules(100, counts=_Tensor(d, i32, 100)), caches=W.kv_caches([_Tensor(d, f32, 1, 20, 64)], [_Kv(d)]))

    class _Kv(_Tensor):
        def __init__(self, d):
            super().__init__(d, f32, 1, 20, 64)

        data_ptr = lambda self: 0x200000  # noqa: E731

    def calls(s, d):
        g = _lib.AttnGeom(1, 1, 64, 64, 64, 0, 0, 1e-6, 0.0)
        r, k, n = _Tensor(d, f32, 3, 64), _Tensor(d, f32, 1, 20, 64), _Tensor(d, i32, 3)
        x, v = _Tensor(d, f32, 3, 100), _Tensor(d, f32, 3)
        return dict(
            rope=lambda: W.rope_axes_rows(s["ax"], [(_Tensor(d, f32, 3, 1, 64), _Tensor(d, f32, 3, 1, 64), None)], s["ws"]),
            attn=lambda: W.attn_tree_sink(g, s["tree"], r, r, r, None, None, None, None, k, k, 5, r, s["ws"]),
            plan=lambda: W.mtp_tree_plan(n, _Tensor(d, i64, 3), n, s["ws"]),
            rules=lambda: W.logit_rules_argmax(s["rules"], x, n, v, None, s["ws"]),
            counts=lambda: W.mtp_token_counts(n, n, False, s["ws"]),
            commit=lambda: W.kv_tree_commit(s["caches"], n, 5, s["ws"]))

    on0 = make(0)
    for name, call in calls(on0, 0).items():
        lib.calls = 0
        call()
        assert lib.calls, name
    current[0] = 1
    on1 = make(1)
    for key, names in dict(ws=("rope", "attn", "plan", "rules", "counts", "commit"), ax=("rope",), tree=("attn",),
                           rules=("rules",), caches=("commit",)).items():
        for name in names:
            lib.calls = 0
            with pytest.raises(ValueError):
                calls({**on1, key: on0[key]}, 1)[name]()
            assert not lib.calls, (key, name)
    with pytest.raises(ValueError):  # a tree whose positions are elsewhere
        W.draft_tree(_Tensor(1, i64, 3), _Tensor(1, i32, 3), on0["ax"])


def test_numbers_past_32_bits_are_refused(monkeypatch):
    """The library takes 32-bit lengths and head strides: a longer one is refused, not cut off."""
    import torch
    from mtp_speculative_draft_gb300 import _lib, tree as W
    i32, i64, f32, u8 = torch.int32, torch.int64, torch.float32, torch.uint8
    lib, big = _Lib(), 1 << 32
    monkeypatch.setattr(W, "_device", lambda: 0)
    monkeypatch.setattr(W, "_on", lambda stream, device: None)
    monkeypatch.setattr(_lib, "load", lambda: lib)
    n, ws, k = _Tensor(0, i32, 3), _Tensor(0, u8, 4096), _Tensor(0, f32, 1, 20, 64)
    v = _Tensor(0, f32, 1, 20, 64)
    v.data_ptr = lambda: 0x200000
    ax = W.rope_axes((32,), _Tensor(0, i32, 1, 3), _Tensor(0, f32, 10, 32, 2))
    tree, caches, r = W.draft_tree(_Tensor(0, i64, 3), n), W.kv_caches([k], [v]), _Tensor(0, f32, 3, 64)
    g = _lib.AttnGeom(1, 1, 64, 64, 64, 0, 0, 1e-6, 0.0)
    wide = _Tensor(0, f32, 3, 2, 64, stride=(64, big + 128, 1))
    for call in (lambda: W.attn_tree_sink(g, tree, r, r, r, None, None, None, None, k, v, big + 5, r, ws),
                 lambda: W.attn_tree_sink_workspace_bytes(g, 3, big + 5),
                 lambda: W.attn_tree_sink_workspace_bytes(g, big + 3, 5),
                 lambda: W.attn_tree_sink(g, tree, r, r, r, None, None, None, None, k, v, 5 - big, r, ws),
                 lambda: W.kv_tree_commit(caches, n, big + 5, ws), lambda: W.kv_tree_commit(caches, n, 5 - big, ws),
                 lambda: W.draft_tree(_Tensor(0, i64, 3), n, None, big),
                 lambda: W.logit_rules(big + 100),
                 lambda: W.logit_rules(100, bias_tokens=_Tensor(0, i32, big + 1), bias=_Tensor(0, f32, big + 1)),
                 lambda: W.logit_rules(100, path_tokens=_Tensor(0, i32, big + 1), path_mask=_Tensor(0, i64, 1)),
                 lambda: W.logit_rules(100, allow=_Tensor(0, i32, 1, big + 4)),
                 lambda: W.logit_rules_argmax_workspace_bytes(big + 4),
                 lambda: W.mtp_token_counts(_Tensor(0, i32, big + 9), n, False, ws),
                 lambda: W.mtp_token_counts(n, _Tensor(0, i32, big + 9), False, ws),
                 lambda: W.mtp_tree_accept(*[_Tensor(0, i32, big + 9)] * 6),
                 lambda: W.mtp_tree_plan(_Tensor(0, i32, big + 9), _Tensor(0, i64, big + 9), _Tensor(0, i32, big + 9), ws),
                 lambda: W.rope_axes((32,), _Tensor(0, i32, 1, big + 3), _Tensor(0, f32, 10, 32, 2)),
                 lambda: W.rope_axes((big + 32,), _Tensor(0, i32, 1, 3), _Tensor(0, f32, big + 32, 2)),
                 lambda: W.rope_axes_rows(ax, [(wide, wide, None)], ws)):
        with pytest.raises(ValueError):
            call()
    assert not lib.calls
    # a longer table is no fault
    assert W.rope_axes((1,), _Tensor(0, i32, 1, 3), _Tensor(0, f32, big + 1, 2)).max_pos == (1 << 31) - 1
