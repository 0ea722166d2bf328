"""The beam search's step on the host: the reference's own pins, workspace sizes, and refusals before anything
reaches a GPU."""

import ctypes as C
import math

import numpy as np
import pytest

from oracle import beam_oracle as B
from oracle import tree_oracle as T

INVALID, UNSUPPORTED, CAPACITY, WORKSPACE, CUDA = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    import torch
    from mtp_speculative_draft_gb300 import build, _lib
    if torch.cuda.is_available():
        pytest.skip("made-up pointers are passed only where no launch can reach a GPU")
    build.build()
    return _lib.load()


# ------------------------------------------------------------------ the reference
@pytest.mark.parametrize("window,sinks", [(0, False), (5, True)])
def test_reference_attention_is_a_chain_over_the_joined_rows(window, sinks):
    rng = np.random.default_rng(1)
    f = lambda *s: rng.standard_normal(s)  # noqa: E731
    nh, nkv, d, dv, m = 4, 2, 8, 6, 3
    plen, tlen = [7, 0], [4, -1, 0, 9]
    q, kn, vn = f(4 * m, nh, d), f(4 * m, nkv, d), f(4 * m, nkv, dv)
    kp, vp, kt, vt = f(2, nkv, 7, d), f(2, nkv, 7, dv), f(4, nkv, 12, d), f(4, nkv, 12, dv)
    s = f(nh) if sinks else None
    out = B.prefix_attention(q, kn, vn, kp, vp, kt, vt, plen, tlen, m, window, s)
    mask, depth = T.tree_plan([-1, 0, 1])
    for b, t in enumerate(tlen):
        rows = slice(b * m, b * m + m)
        if t < 0:
            assert out[rows] == [None] * m
            continue
        P = plen[b // 2]
        joined = [np.concatenate([x[b // 2][:, :P], y[b][:, :t]], 1) for x, y in ((kp, kt), (vp, vt))]
        ref = T.tree_attention(q[rows], *joined, kn[rows], vn[rows], mask, depth, window, s)
        np.testing.assert_allclose(np.array(out[rows]), ref, rtol=1e-12, atol=1e-14)


def test_reference_selection_by_hand():
    # probabilities 1/2, 1/4, 1/4 and 3/4, 1/4, 0
    x = np.log([[0.5, 0.25, 0.25], [0.75, 0.25, 1e-300]])
    x[1, 2] = -np.inf
    s = [math.log(0.4), math.log(0.3)]
    parent, token, score, length, done = B.beam_select(x, 1, 2, 6, s, [3, 3], None, eos=0)
    # 0.225, 0.2, 0.1 (token 1), 0.1 (token 2), 0.075, nothing
    assert parent[0].tolist() == [1, 0, 0, 0, 1, -1] and token[0].tolist() == [0, 0, 1, 2, 1, -1]
    np.testing.assert_allclose(np.exp(score[0]), [0.225, 0.2, 0.1, 0.1, 0.075, 0], rtol=1e-12)
    assert length[0].tolist() == [4] * 5 + [0] and done[0].tolist() == [1, 1, 0, 0, 0, 0]
    # a finished beam of probability 0.3 is carried on as it is; ranks by length: log(0.3) / 3 against log(0.2) / 4
    parent, token, score, length, done = B.beam_select(x, 1, 2, 3, s, [3, 3], [0, 1], eos=2, alpha=1.0)
    assert parent[0].tolist() == [1, 0, 0] and token[0].tolist() == [2, 0, 1]
    assert abs(math.log(0.3) / 3) < abs(math.log(0.1) / 4) and length[0].tolist() == [3, 4, 4] and done[0].tolist() == [1, 0, 0]


def test_reference_selection_of_rows_that_offer_nothing():
    x = np.zeros((4, 5))
    x[0], x[1, 2], x[2, 1] = -np.inf, np.inf, np.nan
    parent, token, _, _, _ = B.beam_select(x, 1, 4, 12, [0.0, 0.0, -1.0, -np.inf])
    assert parent[0].tolist() == [2] * 4 + [-1] * 8 and token[0].tolist() == [0, 2, 3, 4] + [-1] * 8


def test_reference_reorder():
    x = np.arange(4 * 1 * 3 * 1, dtype=float).reshape(4, 1, 3, 1)
    y = B.beam_reorder(x, [[1, 0], [1, -1]], [[2, 3], [1, 3]], 2)
    assert y[:, 0, :, 0].tolist() == [[3, 4, 2], [0, 1, 2], [9, 7, 8], [9, 10, 11]]


# ------------------------------------------------------------------ attn_prefix_sink
P = C.c_void_p(0x1000000)


def _geom(nh=8, nkv=2, dqk=64, dv=64, rot=None, window=0, gated=0, eps=1e-6, scale=0.0):
    from mtp_speculative_draft_gb300 import _lib
    return _lib.AttnGeom(nh, nkv, dqk, dv, dqk if rot is None else rot, window, gated, eps, scale)


def _batch(plen=0x1000, tlen=0x2000, groups=2, seqs=6, m=1, pmax=100, tmax=20, base=0, ldq=0, ldk=0, ldv=0, axes=None):
    from mtp_speculative_draft_gb300 import _lib
    return _lib.PrefixBatch(plen, tlen, axes, groups, seqs, m, pmax, tmax, base, ldq, ldk, ldv)


def _attn(lib, g=None, b=None, ptrs=None, rope_rows=200, pcap=100, tcap=30, ws=0x4000000, ws_bytes=1 << 40, n=None):
    """The call's status; ``ptrs`` replaces pointers by their place (q k v qn kn rope sinks kp vp kt vt out)."""
    p = [P] * 12
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.attn_prefix_sink(C.byref(g or _geom()), C.byref(b or _batch()), *p[:6], rope_rows, *p[6:9], pcap, *p[9:11],
                                tcap, p[11], ws, ws_bytes, None)


def test_attention_refuses(lib):
    odd = C.c_void_p(0x1000004)
    for want, kw in (
            (INVALID, dict(g=_geom(nh=7))), (INVALID, dict(g=_geom(nh=0))), (UNSUPPORTED, dict(g=_geom(nh=130, nkv=65))),
            (UNSUPPORTED, dict(g=_geom(nh=130, nkv=2))), (UNSUPPORTED, dict(g=_geom(dqk=48, rot=32))),
            (UNSUPPORTED, dict(g=_geom(dv=288))), (INVALID, dict(g=_geom(rot=65))), (INVALID, dict(g=_geom(rot=66))),
            (INVALID, dict(g=_geom(gated=2))), (UNSUPPORTED, dict(g=_geom(gated=1, dv=32))),
            (INVALID, dict(g=_geom(eps=float("nan")))), (INVALID, dict(g=_geom(scale=float("inf")))),
            (INVALID, dict(b=_batch(tlen=None))), (UNSUPPORTED, dict(b=_batch(groups=4))), (UNSUPPORTED, dict(b=_batch(groups=0))),
            (UNSUPPORTED, dict(b=_batch(groups=1, seqs=1025))), (UNSUPPORTED, dict(b=_batch(groups=1, seqs=0))),
            (UNSUPPORTED, dict(b=_batch(m=0))), (UNSUPPORTED, dict(b=_batch(m=17))),
            (INVALID, dict(b=_batch(pmax=-1))), (INVALID, dict(b=_batch(tmax=-1))), (CAPACITY, dict(b=_batch(pmax=101))),
            (CAPACITY, dict(b=_batch(tmax=30))), (CAPACITY, dict(b=_batch(tmax=2 ** 31 - 1))), (CAPACITY, dict(b=_batch(tmax=15, m=16))),
            (INVALID, dict(b=_batch(plen=None))), (INVALID, dict(ptrs={0: None})), (INVALID, dict(ptrs={7: None})),
            (INVALID, dict(ptrs={9: None})), (INVALID, dict(ptrs={11: None})), (INVALID, dict(ptrs={5: None})),
            (INVALID, dict(ptrs={6: C.c_void_p(0x1000002)})), (INVALID, dict(b=_batch(tlen=0x2002))),
            (INVALID, dict(rope_rows=120)), (INVALID, dict(b=_batch(base=-1))), (INVALID, dict(b=_batch(base=2 ** 31 - 1))),
            (INVALID, dict(b=_batch(ldq=508))), (INVALID, dict(b=_batch(ldk=130))), (INVALID, dict(b=_batch(ldv=-4))),
            (INVALID, dict(pcap=-1)), (INVALID, dict(tcap=0)),
            (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=0x4000008)), (WORKSPACE, dict(ws_bytes=2000))):
        assert _attn(lib, **kw) == want, kw
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 9, 10, 11):
        assert _attn(lib, ptrs={i: odd}) == INVALID, i


def test_attention_takes_no_prompt_without_pointers_up_to_the_workspace(lib):
    """Prompts of no rows need no arrays; nothing else is missing, so the workspace is what is refused."""
    assert _attn(lib, b=_batch(plen=None, pmax=0), ptrs={7: None, 8: None}, pcap=0, ws_bytes=0) == WORKSPACE
    assert _attn(lib, g=_geom(rot=0), ptrs={5: None}, rope_rows=0, ws_bytes=0) == WORKSPACE


@pytest.mark.parametrize("nh,nkv,dqk,dv,window", [(40, 8, 128, 128, 0), (16, 2, 256, 256, 0), (4, 2, 64, 64, 0),
                                                  (32, 8, 192, 128, 128), (64, 1, 32, 256, 0), (7, 1, 96, 32, 3000)])
def test_workspace_of_the_largest_call_does_for_all(lib, nh, nkv, dqk, dv, window):
    """The size grows with prompts, sequences, rows and the prompts' length."""
    g = _geom(nh, nkv, dqk, dv, window=window)
    size = lambda *a: lib.attn_prefix_sink_workspace_bytes(C.byref(g), *a)  # noqa: E731
    lengths = [0, 1, 64, 65, 127, 128, 129, 300, 1000, 4095, 4096, 4097, 32768]
    for groups, per, m in ((1, 1, 1), (1, 7, 2), (2, 3, 1), (3, 20, 5), (1, 64, 1), (4, 16, 16), (1, 1024, 1), (8, 128, 3)):
        at = [size(groups, groups * per, m, L) for L in lengths]
        assert all(a <= b for a, b in zip(at, at[1:]))
        for L, need in zip(lengths, at):
            assert need <= size(groups, groups * per, min(16, m + 1), L)
            if (per + 1) * groups <= 1024:
                assert need <= size(groups, groups * (per + 1), m, L)
            if per * (groups + 1) <= 1024:
                assert need <= size(groups + 1, (groups + 1) * per, m, L)
            # no call of that size or of a smaller one, with tails of any length, is refused its workspace (it then
            # fails for want of a GPU)
            for groups2, per2, m2, L2, tmax in ((groups, per, m, L, 20), (groups, per, m, L, 5000), (1, max(1, per // 2), m, L, 40000),
                                                (1, 1, 1, L, 100000), (groups, per, 1, L // 2, 300), (1, max(1, per // 3), 1, L, 3000)):
                b = _batch(groups=groups2, seqs=groups2 * per2, m=m2, pmax=L2, tmax=tmax)
                call = lambda n: _attn(lib, g, b, pcap=40000, tcap=200000, rope_rows=200000, ws_bytes=n)  # noqa: E731
                assert call(18000) == WORKSPACE and call(need) == CUDA, (groups2, per2, m2, L2, tmax)
    for bad in ((0, 1, 1, 5), (2, 3, 1, 5), (1, 1025, 1, 5), (1, 4, 17, 5), (1, 4, 1, -1)):
        assert size(*bad) == 0
    assert lib.attn_prefix_sink_workspace_bytes(None, 1, 1, 1, 5) == 0
    odd = _geom(3, 2)
    assert lib.attn_prefix_sink_workspace_bytes(C.byref(odd), 1, 1, 1, 5) == 0


# ------------------------------------------------------------------ beam_select
def _set(score=0x1000, length=0x2000, done=0x3000, seqs=2, beams=4, vocab=100, eos=2, alpha=1.0):
    from mtp_speculative_draft_gb300 import _lib
    return _lib.BeamSet(score, length, done, seqs, beams, vocab, eos, alpha)


def _select(lib, s=None, x=0x100000, ld=100, k=4, parent=0x4000, token=0x5000, score=0x6000, length=0x7000, done=0x8000,
            ws=0x9000000, ws_bytes=1 << 40):
    return lib.beam_select(C.byref(s or _set()), x, ld, k, parent, token, score, length, done, ws, ws_bytes, None)


def test_selection_refuses(lib):
    for want, kw in (
            (INVALID, dict(s=_set(score=None))), (INVALID, dict(x=None)), (INVALID, dict(parent=None)),
            (INVALID, dict(token=None)), (INVALID, dict(score=None)),
            (UNSUPPORTED, dict(s=_set(seqs=0))), (UNSUPPORTED, dict(s=_set(beams=0))), (UNSUPPORTED, dict(s=_set(beams=65))),
            (UNSUPPORTED, dict(s=_set(seqs=257))), (UNSUPPORTED, dict(s=_set(seqs=2 ** 30, beams=4))),
            (UNSUPPORTED, dict(s=_set(vocab=0, eos=-1, done=None))), (UNSUPPORTED, dict(s=_set(vocab=2 ** 30 + 1), ld=2 ** 31)),
            (UNSUPPORTED, dict(k=0)), (UNSUPPORTED, dict(k=129)), (INVALID, dict(ld=99)),
            (INVALID, dict(s=_set(eos=100))), (INVALID, dict(s=_set(eos=-1))), (INVALID, dict(s=_set(eos=-2, done=None))),
            (INVALID, dict(s=_set(alpha=float("nan")))), (INVALID, dict(s=_set(length=None))),
            (INVALID, dict(s=_set(length=None, alpha=0.0))),
            (INVALID, dict(s=_set(score=0x1002))), (INVALID, dict(x=0x100001)), (INVALID, dict(done=0x8001)),
            (INVALID, dict(score=0x1000, k=3)),            # in place with fewer candidates than beams
            (INVALID, dict(score=0x1004)),                 # overlaps its input by a part
            (INVALID, dict(length=0x3000)),                # new lengths into the old flags
            (INVALID, dict(parent=0x5004)),                # outputs overlap
            (INVALID, dict(token=0x100000 + 4 * 799)),     # the last logit
            (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=0x9000004)), (WORKSPACE, dict(ws_bytes=18000))):
        assert _select(lib, **kw) == want, kw
    # in place, and an output right behind the logits, are fine: only the workspace is missing
    assert _select(lib, score=0x1000, length=0x2000, done=0x3000, ws=None) == WORKSPACE
    assert _select(lib, token=0x100000 + 4 * 800, ws=None) == WORKSPACE
    assert _select(lib, s=_set(length=None, done=None, alpha=0.0, eos=-1), length=None, done=None, ws=None) == WORKSPACE


def test_selection_workspace(lib):
    size = lib.beam_select_workspace_bytes
    for bad in ((0, 4, 100, 4), (1, 65, 100, 4), (17, 64, 100, 4), (1, 4, 0, 4), (1, 4, 100, 129), (-1, 4, 100, 4)):
        assert size(*bad) == 0
    for a, b in (((1, 4, 100, 4), (2, 4, 100, 4)), ((1, 4, 100, 4), (1, 4, 100, 5)), ((3, 4, 9000, 4), (3, 4, 90000, 4)),
                 ((3, 4, 9000, 4), (3, 5, 9000, 4))):
        assert 0 < size(*a) <= size(*b)
    need = size(2, 4, 100, 4)
    assert _select(lib, ws_bytes=need - 1) == WORKSPACE


# ------------------------------------------------------------------ kv_beam_reorder
def _caches(layers=2, nkv=2, dqk=64, dv=32, cap=50, k=0x10000, v=0x20000):
    from mtp_speculative_draft_gb300 import _lib
    ks, vs = (C.c_void_p * layers)(*[k] * layers), (C.c_void_p * layers)(*[v] * layers)
    c = _lib.KvCaches(ks, vs, layers, nkv, dqk, dv, cap)
    c.keep = ks, vs
    return c


def _reorder(lib, c=None, parent=P, seqs=2, beams=4, length=P, most=50, ws=0x9000000, ws_bytes=1024):
    return lib.kv_beam_reorder(C.byref(c or _caches()), parent, seqs, beams, length, most, ws, ws_bytes, None)


def test_reorder_refuses(lib):
    for want, kw in (
            (INVALID, dict(parent=None)), (INVALID, dict(length=None)), (INVALID, dict(parent=C.c_void_p(0x1002))),
            (UNSUPPORTED, dict(seqs=0)), (UNSUPPORTED, dict(beams=65)), (UNSUPPORTED, dict(seqs=300)),
            (UNSUPPORTED, dict(seqs=2 ** 31 - 1)), (UNSUPPORTED, dict(c=_caches(nkv=65))), (UNSUPPORTED, dict(c=_caches(dqk=6))),
            (UNSUPPORTED, dict(c=_caches(dv=260))), (INVALID, dict(most=-1)), (CAPACITY, dict(most=51)),
            (INVALID, dict(c=_caches(k=None))), (INVALID, dict(c=_caches(v=0x20008))),
            (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=0x9000004)), (WORKSPACE, dict(ws_bytes=1000))):
        assert _reorder(lib, **kw) == want, kw
    assert _reorder(lib, most=0) == 0  # no row moves: nothing is launched
    assert lib.kv_beam_workspace_bytes() == 1024


def test_caches_of_one_layout_are_refused_where_the_other_is_taken(monkeypatch):
    """Caches [n_kv, cap, dim] and beams' tails [rows, n_kv, cap, dim] have one descriptor: each call takes its own."""
    import torch
    from mtp_speculative_draft_gb300 import _lib, beams as W, tree as T_
    from test_tree_calls_host import _Lib, _Tensor
    lib, at = _Lib(), iter(range(0x100000, 0x900000, 0x100000))
    for m in (W, T_):
        monkeypatch.setattr(m, "_device", lambda: 0)
        monkeypatch.setattr(m, "_on", lambda stream, device: None)
    monkeypatch.setattr(_lib, "load", lambda: lib)

    def cache(*shape):
        t = _Tensor(0, torch.float32, *shape)
        p = next(at)
        t.data_ptr = lambda: p
        return t

    n, ws = _Tensor(0, torch.int32, 4), _Tensor(0, torch.uint8, 4096)
    caches = T_.kv_caches([cache(2, 20, 64)], [cache(2, 20, 64)])
    tails = W.kv_tails([cache(4, 2, 20, 64)], [cache(4, 2, 20, 64)], 2)
    T_.kv_tree_commit(caches, n, 5, ws)
    W.kv_beam_reorder(tails, n, n, 5, ws)
    assert lib.calls == 2
    for call in (lambda: T_.kv_tree_commit(tails, n, 5, ws), lambda: W.kv_beam_reorder(caches, n, n, 5, ws)):
        with pytest.raises(ValueError):
            call()
    assert lib.calls == 2
    # a descriptor that a program filled in by itself goes to the call it was made for
    own = _lib.KvCaches(caches.h_k, caches.h_v, 1, 2, 64, 64, 20)
    T_.kv_tree_commit(own, n, 5, ws)
    own.seqs, own.beams = 2, 2
    W.kv_beam_reorder(own, n, n, 5, ws)
    assert lib.calls == 4


@pytest.fixture(scope="module")
def move_plan(tmp_path_factory):
    """The tiles of kv_beam_reorder, compiled so that undefined arithmetic ends the program: (shift, rows, tiles) of
    lines "beams wide lists max_len sms"."""
    import os
    import shutil
    import subprocess
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("move")
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mtp_speculative_draft_gb300", "csrc")
    (at / "plan.cpp").write_text('#include <cstdio>\n#include "move.h"\n'
                                 "int main() {\n  int b, w, m, s;\n  long long l;\n"
                                 '  while (scanf("%d %d %lld %d %d", &b, &w, &l, &m, &s) == 5) {\n'
                                 "    const mtp::MovePlan p = mtp::move_plan(b, w, l, m, s);\n"
                                 '    printf("%d %d %lld\\n", p.shift, p.rows, (long long)p.tiles);\n  }\n}\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", csrc,
                    str(at / "plan.cpp"), "-o", str(at / "plan")], check=True)

    def run(cases):
        done = subprocess.run([str(at / "plan")], input="".join("%d %d %d %d %d\n" % c for c in cases), capture_output=True,
                              text=True)
        assert done.returncode == 0, done.stderr
        plans = [tuple(map(int, line.split())) for line in done.stdout.splitlines()]
        assert len(plans) == len(cases)
        for (beams, wide, _, most, _), (shift, rows, tiles) in zip(cases, plans):
            # the beams' tiles fit the CTA's registers, and the tiles cover the rows, each with some
            assert shift >= 0 and beams << shift <= 4096 and 1 <= rows and rows * wide <= 4 << shift
            assert (tiles - 1) * rows < most <= tiles * rows
        return plans

    return run


def test_tiles_of_the_narrowest_rows(move_plan):
    """Rows of 4 dims and few lists: tiles shrink to one 16-byte word a beam, and no further."""
    cases = [(b, w, n, most, 152) for b in (1, 2, 3, 5, 17, 64) for w in (4, 8, 12, 64, 256) for n in (1, 2, 16, 4096)
             for most in (1, 2, 17, 100, 4096)]
    plans = move_plan(cases)
    assert plans[cases.index((1, 4, 1, 1, 152))] == (0, 1, 1)


def test_tiles_of_tails_near_the_longest_length(move_plan):
    """Bounds up to 2^31 - 1 rows: the rounding up to whole tiles passes 32 bits."""
    most = 2 ** 31 - 1
    plans = move_plan([(b, w, n, m, 152) for b in (1, 2, 64) for w in (4, 64, 256) for n in (1, 4096) for m in (most, most - 1, 2 ** 30 + 1)])
    assert plans[0] == (12, 4096, 2 ** 19)
