"""Draft-tree calls: descriptors match the header, and invalid calls are refused on the host before
anything reaches a GPU; the float64 reference against hand-worked cases."""

import ctypes as C
import os
import subprocess
import tempfile

import numpy as np
import pytest

from oracle import mtp_oracle as O
from oracle import tree_oracle as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = C.c_void_p(0x100000)


@pytest.fixture(scope="module")
def lib():
    from mtp_speculative_draft_gb300 import build, _lib
    build.build()
    return _lib.load()


def test_struct_layouts_match_c(lib):
    from mtp_speculative_draft_gb300 import _lib
    src = r'''
    #include <stdio.h>
    #include <stddef.h>
    #include "mtpdraft.h"
    int main(void) {
      printf("%zu %zu %zu %zu %zu\n", sizeof(mtp_rope_axes), sizeof(mtp_head_rows),
             sizeof(mtp_draft_tree), sizeof(mtp_logit_rules), sizeof(mtp_kv_caches));
      printf("%zu %zu %zu %zu %zu\n", offsetof(mtp_rope_axes, max_pos), offsetof(mtp_head_rows, n_heads),
             offsetof(mtp_draft_tree, ld_v), offsetof(mtp_logit_rules, n_path),
             offsetof(mtp_kv_caches, cache_cap));
      return 0; }
    '''
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    s = (_lib.RopeAxes, _lib.HeadRows, _lib.DraftTree, _lib.LogitRules, _lib.KvCaches)
    assert got == [C.sizeof(x) for x in s] + [_lib.RopeAxes.max_pos.offset, _lib.HeadRows.n_heads.offset,
                                              _lib.DraftTree.ld_v.offset, _lib.LogitRules.n_path.offset,
                                              _lib.KvCaches.cache_cap.offset]


# ------------------------------------------------------------------ refusals
def _axes(sections=(24, 20, 20), inter=1, n=None, pos_ld=8, max_pos=100, pos=0x1000, rope=0x2000):
    from mtp_speculative_draft_gb300 import _lib
    sec = list(sections) + [0] * (4 - len(sections))
    return _lib.RopeAxes(pos, rope, len(sections) if n is None else n, (C.c_int32 * 4)(*sec), inter, pos_ld, max_pos)


def test_rope_axes_rows_refusals(lib):
    from mtp_speculative_draft_gb300 import _lib

    def call(ax=None, rows=4, d=128, x=0x10000, y=0x20000, hs=128, ld=1024, heads=8, ws=P, wsb=1024, eps=1e-6, nt=1):
        ax = _axes() if ax is None else ax
        t = (_lib.HeadRows * 1)(_lib.HeadRows(x, y, None, ld, 1024, hs, 128, heads))
        return lib.rope_axes_rows(C.byref(ax), t, nt, rows, d, eps, ws, wsb, None)

    assert call(rows=0) == 1 and call(rows=9) == 1       # no rows; more rows than positions
    assert call(d=48) == 2 and call(d=288) == 2          # head size
    assert call(x=None) == 1 and call(x=0x10004) == 1    # null, misaligned
    assert call(hs=96) == 1 and call(ld=1000) == 1       # overlapping heads, rows
    assert call(hs=130, ld=1042) == 1                    # strides not multiples of 4
    assert call(x=0x20000, ld=1028) == 1                 # in place with another stride
    assert call(heads=0) == 2 and call(nt=0) == 1 and call(nt=5) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(ws=None) == 4 and call(wsb=1000) == 4
    assert call(_axes(n=0)) == 2 and call(_axes(n=5)) == 2
    assert call(_axes(pos=None)) == 1 and call(_axes(rope=None)) == 1
    assert call(_axes((64, 64, 64))) == 1                # 192 pairs
    assert call(_axes((40, 40, 0), inter=0), d=128) == 1  # 80 pairs in a head of 128
    assert call(_axes((0, 40, 24))) == 1                 # interleaved: axis 1 has 21 turns in 64 pairs
    assert call(_axes(inter=2)) == 1 and call(_axes(max_pos=0)) == 1 and call(_axes((-1, 33, 32))) == 1


def test_attn_tree_refusals(lib):
    from mtp_speculative_draft_gb300 import _lib

    def call(g=(8, 2, 128, 128, 128, 0, 0, 1e-6, 0.0), n=4, L=10, cap=64, q=0x10000, mask=0x1000, depth=0x2000,
             rows=64, wsb=None, ws=P, base=0, axes=None, ld=0, rope=0x30000):
        geo = _lib.AttnGeom(*g)
        t = _lib.DraftTree(mask, depth, C.pointer(axes) if axes is not None else None, n, base, ld, 0, 0)
        need = lib.attn_tree_sink_workspace_bytes(C.byref(geo), max(1, min(n, 64)), max(0, L))
        return lib.attn_tree_sink(C.byref(geo), C.byref(t), q, 0x20000, 0x30000, None, None, rope, rows, None,
                                  0x40000, 0x50000, L, cap, 0x60000, ws, need if wsb is None else wsb, None)

    assert call(n=0) == 2 and call(n=65) == 2
    assert call(q=None) == 1 and call(q=0x10004) == 1 and call(mask=None) == 1 and call(depth=None) == 1
    assert call(mask=0x1004) == 1
    assert call(g=(8, 3, 128, 128, 128, 0, 0, 1e-6, 0.0)) == 1    # heads that do not group
    assert call(g=(130, 2, 128, 128, 128, 0, 0, 1e-6, 0.0)) == 2  # 65 query heads a KV head
    assert call(g=(8, 2, 144, 128, 128, 0, 0, 1e-6, 0.0)) == 2    # head size
    assert call(g=(8, 2, 128, 64, 128, 0, 1, 1e-6, 0.0)) == 2     # gate with another value size
    assert call(g=(8, 2, 128, 128, 127, 0, 0, 1e-6, 0.0)) == 1    # odd rotation
    assert call(g=(8, 2, 128, 128, 128, 0, 0, 1e-6, -1.0)) == 1   # negative scale
    assert call(L=-1) == 1 and call(L=61) == 3 and call(L=2 ** 31 - 2, cap=2 ** 31 - 1) == 3
    assert call(rows=13) == 1 and call(base=51) == 1 and call(base=-1) == 1 and call(rope=None) == 1
    assert call(ld=1000) == 1 and call(ld=1026) == 1
    assert call(axes=_axes((16, 8, 8))) == 1                      # 32 pairs, rot_dim / 2 is 64
    assert call(axes=_axes(pos_ld=3)) == 1
    assert call(ws=None) == 4 and call(wsb=1024) == 4


def test_logit_rules_refusals(lib):
    from mtp_speculative_draft_gb300 import _lib

    def call(rows=4, ld=1000, ldo=1000, x=0x10000, out=None, wsb=4096, tok=P, **kw):
        f = dict(vocab=1000, repetition=1.0, frequency=0.0, presence=0.0, d_counts=None, d_bias_tokens=None,
                 d_bias=None, n_bias=0, d_allow=None, allow_ld=0, d_path_tokens=None, d_path_mask=None, n_path=0)
        f.update(kw)
        r = _lib.LogitRules(*f.values())
        return lib.logit_rules_argmax(C.byref(r), x, ld, rows, tok, P, out, ldo, P, wsb, None)

    assert call(x=None) == 1 and call(tok=None) == 1
    assert call(rows=0) == 2 and call(rows=1025) == 2 and call(vocab=0) == 2
    assert call(ld=999) == 1 and call(out=0x90000, ldo=999) == 1
    assert call(out=0x10000, ldo=1004) == 1                       # in place with another stride
    assert call(repetition=0.0) == 1 and call(repetition=float("inf")) == 1 and call(repetition=float("nan")) == 1
    assert call(presence=float("inf")) == 1 and call(frequency=float("nan")) == 1
    assert call(n_bias=3) == 1 and call(n_bias=-1) == 1 and call(n_bias=65537) == 1
    assert call(n_path=3) == 1 and call(n_path=65, d_path_tokens=0x1000, d_path_mask=0x1000) == 1
    assert call(d_allow=0x1000, allow_ld=31) == 1
    assert call(d_path_tokens=0x1000, d_path_mask=0x1004, n_path=2) == 1
    assert call(x=0x10002) == 1 and call(d_allow=0x1001, allow_ld=32) == 1
    assert call(wsb=1024) == 4
    assert lib.logit_rules_argmax_workspace_bytes(0) == 0
    assert lib.mtp_token_counts(None, 10, P, 3, 0, P, 1024, None) == 1
    assert lib.mtp_token_counts(P, 10, P, 0, 0, P, 1024, None) == 1
    assert lib.mtp_token_counts(P, 10, P, 3, 2, P, 1024, None) == 1
    assert lib.mtp_token_counts(P, 10, P, 3, 0, P, 100, None) == 4


def test_tree_refusals(lib):
    from mtp_speculative_draft_gb300 import _lib
    assert lib.mtp_tree_plan(P, 0, P, P, P, 1024, None) == 2 and lib.mtp_tree_plan(P, 65, P, P, P, 1024, None) == 2
    assert lib.mtp_tree_plan(None, 4, P, P, P, 1024, None) == 1
    assert lib.mtp_tree_plan(P, 4, C.c_void_p(0x1004), P, P, 1024, None) == 1
    assert lib.mtp_tree_plan(P, 4, P, P, P, 100, None) == 4
    assert lib.mtp_tree_accept(P, P, None, 4, P, P, P, None) == 1
    assert lib.mtp_tree_accept(P, P, P, 65, P, P, P, None) == 2

    def commit(n=4, L=0, cap=64, nkv=2, d=64, k=0x1000, layers=1, wsb=1024):
        ks, vs = (C.c_void_p * 1)(k), (C.c_void_p * 1)(0x2000)
        c = _lib.KvCaches(ks, vs, layers, nkv, d, d, cap)
        return lib.kv_tree_commit(C.byref(c), P, n, L, P, wsb, None)

    assert commit(n=0) == 2 and commit(n=65) == 2 and commit(L=61) == 3 and commit(L=-1) == 1
    assert commit(nkv=0) == 2 and commit(d=66) == 2 and commit(d=260) == 2 and commit(layers=0) == 2
    assert commit(k=None) == 1 and commit(k=0x1004) == 1 and commit(wsb=1000) == 4


def test_wrappers_refuse_host_tensors():
    import torch
    from mtp_speculative_draft_gb300 import draft_tree, kv_caches, logit_rules, rope_axes
    z = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: rope_axes((8,), z.view(1, 4), torch.zeros(64)), lambda: logit_rules(10, counts=z),
                 lambda: draft_tree(torch.zeros(4, dtype=torch.int64), z),
                 lambda: kv_caches([torch.zeros(1, 4, 32)], [torch.zeros(1, 4, 32)])):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the float64 reference
def test_reference_axes():
    assert T.axis_of_pair((3, 1, 2), False) == [0, 0, 0, 1, 2, 2]
    assert T.axis_of_pair((24, 20, 20), True)[:7] == [0, 1, 2, 0, 1, 2, 0]
    assert [T.axis_of_pair((24, 20, 20), True).count(a) for a in range(3)] == [24, 20, 20]
    # equal positions on every axis: the one-axis rotation of the draft layer
    x = np.random.default_rng(0).standard_normal((3, 2, 64))
    got = T.rope_axes(x, [[5, 9, 11]] * 3, (12, 10, 10), True, 1e6)
    for r, p in enumerate((5, 9, 11)):
        np.testing.assert_allclose(got[r], [O.rope(h, p, 1e6, 64) for h in x[r]], rtol=0, atol=1e-12)


def test_reference_attention_of_a_chain_is_causal():
    rng = np.random.default_rng(1)
    n, nh, nkv, d, L = 3, 4, 2, 32, 5
    q, kn, vn = rng.standard_normal((n, nh, d)), rng.standard_normal((n, nkv, d)), rng.standard_normal((n, nkv, d))
    kc, vc = rng.standard_normal((nkv, L, d)), rng.standard_normal((nkv, L, d))
    mask, depth = T.tree_plan([-1, 0, 1])
    got = T.tree_attention(q, kc, vc, kn, vn, mask, depth, window=4)
    for i in range(n):
        for h in range(nh):
            K = np.concatenate([kc[h // 2], kn[:, h // 2]])[max(0, L + i - 3):L + i + 1]
            V = np.concatenate([vc[h // 2], vn[:, h // 2]])[max(0, L + i - 3):L + i + 1]
            p = np.exp(K @ q[i, h] / np.sqrt(d))
            np.testing.assert_allclose(got[i, h], p @ V / p.sum(), rtol=1e-12)
    assert not T.tree_attention(q, kc[:, :0], vc[:, :0], kn, vn, [0, 1, 3], depth)[0].any()  # sees nothing


def test_reference_rules_and_accept():
    l = np.array([[2.0, -2.0, 1.0, 0.5]])
    got = T.logit_rules(l, counts=[1, 2, 0x80000000, 0], repetition=2.0, frequency=0.5, presence=0.25,
                        bias=[(3, 1.0), (3, 2.0), (9, 5.0)], allow=[0b1011], path_tokens=[1, 3], path_mask=[0b01])
    # token 0: 2/2 - .5 - .25; token 1: -2*2 - 3*.5 - .25; token 2 in the prompt only, forbidden; token 3: .5 + 3
    np.testing.assert_allclose(got, [[0.25, -5.75, -np.inf, 3.5]])
    assert T.greedy(got) == [(3, 3.5)]
    assert T.greedy([np.array([np.nan, -np.inf])]) == [(-1, -np.inf)]
    # two children match: the lower one is taken, though only the other has a matching child
    path, emitted = T.tree_accept([-1, 0, 0, 2, 3], [9, 4, 4, 5, 6], [4, 7, 5, 6, 8])
    assert (path, emitted) == ([0, 1], [4, 7])
    path, emitted = T.tree_accept([-1, 0, 0, 2, 3], [9, 3, 4, 5, 6], [4, 7, 5, 6, 8])
    assert (path, emitted) == ([0, 2, 3, 4], [4, 5, 6, 8])
