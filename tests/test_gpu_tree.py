"""Draft-tree operators on the GPU against the float64 reference.

Tolerances (errors scaled by max(|ref|, rms(ref)), as in helpers.py):

* rotation: a normalised value takes at most 6 float32 roundings (square sum's last step, the root's two
  units, two products, the table's rounding) and a rotated one 3 more, each at most 2^-24 of a value no
  larger than sqrt(2) times the pair: 9 * 1.5 * 2^-24 = 8e-7, doubled for the sum of squares' own error: 2e-6.
* attention: a logit is a sum of d products of order |q||k| / d each; with operands of at least 22 bits its
  error is about sqrt(d) * 2^-22 * 0.3 (random signs) plus 9 roundings of q and k: below 2e-6 absolute for
  d <= 256 and logits of order 5 (six standard deviations).  A weight moves by twice that, the output by at
  most 2 * 2e-6 * max|v| (about 4) = 1.6e-5; the bound is 3e-5.
* rules, accept, commit: bit for bit.
"""

import numpy as np
import pytest

from helpers import assert_close
from oracle import tree_oracle as T

pytestmark = pytest.mark.gpu

ROPE_TOL, ATTN_TOL = 2e-6, 3e-5


@pytest.fixture(scope="module")
def dev():
    import torch
    from mtp_speculative_draft_gb300 import build
    build.build()
    torch.cuda.init()
    return torch.device("cuda:0")


def _t(a, dev):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _words(mask, dev):
    return _t(np.array([int(m) for m in mask], dtype=np.uint64).view(np.int64), dev)


def _parents(rng, n, kind):
    if kind == "chain":
        return [-1] + list(range(n - 1))
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "forest":
        return [-1 if i % 5 == 0 else int(rng.integers(max(0, i - 4), i)) for i in range(n)]
    return [-1] + [int(rng.integers(max(0, i - 9), i)) for i in range(1, n)]


def _table(max_pos, rot, theta, dev):
    import torch
    from mtp_speculative_draft_gb300 import mtp_rope_table
    t = torch.empty(max(1, max_pos * rot), dtype=torch.float32, device=dev)
    if rot:
        mtp_rope_table(t, max_pos, rot, theta)
    return t


# ------------------------------------------------------------------ rope_axes_rows
@pytest.mark.parametrize("rows,nh,nkv,d,sections,inter,norm,pad,gated", [
    (1, 40, 8, 128, (24, 20, 20), True, True, 0, True),
    (1, 1, 1, 32, (1,), False, False, 0, False),
    (7, 4, 2, 64, (32,), False, True, 4, False),
    (65, 6, 3, 96, (5, 5, 5), True, True, 12, False),       # rot 30: pairs not in quads
    (33, 3, 1, 160, (16, 0, 24), False, False, 0, False),   # an empty section, dims past the rotation
    (130, 2, 2, 256, (44, 42, 42), True, True, 0, True),
    (17, 5, 5, 224, (4, 4, 4, 4), True, True, 0, False),    # four axes, rot 32 of 224
    (3, 17, 1, 32, (8, 8), False, True, 0, False),
])
def test_rope_axes_rows(dev, rows, nh, nkv, d, sections, inter, norm, pad, gated):
    import torch
    from mtp_speculative_draft_gb300 import mtp_workspace_status, rope_axes, rope_axes_rows
    rng = np.random.default_rng(rows * 100 + d)
    rot, max_pos, n = 2 * sum(sections), 500, len(sections)
    pos = rng.integers(0, max_pos, (n, rows + 3)).astype(np.int32)
    pos[:, 0] = max_pos - 1
    width = (2 if gated else 1) * d
    q = rng.standard_normal((rows, nh * width + pad)).astype(np.float32)
    k = rng.standard_normal((rows, nkv, d)).astype(np.float32)
    qn = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32) if norm else None
    tq = _t(q, dev)[:, :nh * width].unflatten(1, (nh, width))[..., :d]
    tk = _t(k, dev)
    yq = torch.full((rows, nh, d), 7.0, device=dev)
    ax = rope_axes(sections, _t(pos, dev), _table(max_pos, rot, 1e4, dev), interleaved=inter)
    ws = rope_axes_rows(ax, [(tq, yq, _t(qn, dev)), (tk, tk, None)])  # k in place
    torch.cuda.synchronize()
    assert mtp_workspace_status(ws) == 0
    qv = q[:, :nh * width].reshape(rows, nh, width)[..., :d]
    ref = T.rope_axes(T.head_norm(qv, qn, 1e-6), pos, sections, inter, 1e4)
    assert_close(yq.cpu().numpy(), ref, "q", ROPE_TOL)
    assert_close(tk.cpu().numpy(), T.rope_axes(k, pos, sections, inter, 1e4), "k", ROPE_TOL)


def test_rope_position_outside_the_table(dev):
    import torch
    from mtp_speculative_draft_gb300 import (mtp_workspace_status, rope_axes, rope_axes_rows, workspace)
    x = torch.randn(3, 2, 64, device=dev)
    y = torch.empty_like(x)
    ax = rope_axes((32,), torch.tensor([[4, -1, 10]], dtype=torch.int32, device=dev), _table(10, 64, 1e4, dev))
    ws = workspace(1024)
    rope_axes_rows(ax, [(x, y, None)], ws)
    torch.cuda.synchronize()
    assert mtp_workspace_status(ws) == 6
    ref = T.rope_axes(x.cpu().numpy(), [[4, 0, 0]], (32,), False, 1e4)  # position 0 is used
    assert_close(y.cpu().numpy(), ref, "rows", ROPE_TOL)


# ------------------------------------------------------------------ attn_tree_sink
def _attn_case(seed, nh, nkv, dqk, dv, L, n, rot=None, window=0, gated=False, norm=True, sinks=False, tree="random",
               axes=None, pos_base=0, cap_extra=3):
    rng = np.random.default_rng(seed)
    rot = dqk if rot is None else rot
    c = dict(nh=nh, nkv=nkv, dqk=dqk, dv=dv, L=L, n=n, rot=rot, window=window, gated=gated, axes=axes,
             pos_base=pos_base, cap=L + n + cap_extra, theta=1e4)
    c["parents"] = _parents(rng, n, tree)
    c["mask"], c["depth"] = T.tree_plan(c["parents"])
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    c["qp"], c["kp"], c["vp"] = f(n, nh * dqk * (2 if gated else 1)), f(n, nkv * dqk), f(n, nkv * dv)
    c["kc"], c["vc"] = f(nkv, L, dqk), f(nkv, L, dv)
    c["qn"], c["kn"] = (1 + 0.1 * f(dqk), 1 + 0.1 * f(dqk)) if norm else (None, None)
    c["sinks"] = f(nh) if sinks else None
    c["pos"] = rng.integers(0, 300, (len(axes), n)).astype(np.int32) if axes else None
    return c


def _reference(c):
    n, nh, nkv, dqk, dv, L = (c[k] for k in ("n", "nh", "nkv", "dqk", "dv", "L"))
    raw = c["qp"].reshape(n, nh, -1)
    sec = c["axes"] or (c["rot"] // 2,)
    pos = c["pos"] if c["axes"] else [[c["pos_base"] + L + d for d in c["depth"]]]
    turn = (lambda x: T.rope_axes(x, pos, sec, True, c["theta"])) if c["rot"] else (lambda x: np.asarray(x, np.float64))
    q = turn(T.head_norm(raw[..., :dqk], c["qn"], 1e-6))
    k = turn(T.head_norm(c["kp"].reshape(n, nkv, dqk), c["kn"], 1e-6))
    v = c["vp"].reshape(n, nkv, dv)
    out = T.tree_attention(q, c["kc"], c["vc"], k, v, c["mask"], c["depth"], c["window"], c["sinks"],
                           raw[..., dqk:] if c["gated"] else None)
    return out.reshape(n, nh * dv), k, v


class Call:
    """Device copies of a case's inputs and its call."""

    def __init__(self, c, dev, pad=0):
        import torch
        from mtp_speculative_draft_gb300 import attn_geom, attn_tree_sink_workspace_bytes, draft_tree, rope_axes, workspace
        self.c, nkv, L, cap = c, c["nkv"], c["L"], c["cap"]
        strided = lambda a: _t(np.pad(a, ((0, 0), (0, pad)), constant_values=np.nan), dev)[:, :a.shape[1]]  # noqa: E731
        self.qp, self.kp, self.vp = strided(c["qp"]), strided(c["kp"]), strided(c["vp"])
        # rows past the tree's hold NaN and have to stay as they are
        self.k = torch.full((nkv, cap, c["dqk"]), float("nan"), device=dev)
        self.v = torch.full((nkv, cap, c["dv"]), float("nan"), device=dev)
        self.k[:, :L], self.v[:, :L] = _t(c["kc"], dev), _t(c["vc"], dev)
        self.qn, self.kn, self.sinks = _t(c["qn"], dev), _t(c["kn"], dev), _t(c["sinks"], dev)
        self.g = attn_geom(c["nh"], nkv, c["dqk"], c["dv"], c["rot"], c["window"], c["gated"])
        axes = None
        if c["axes"]:
            axes = rope_axes(c["axes"], _t(c["pos"], dev), _table(300, c["rot"], c["theta"], dev), interleaved=True)
        self.tree = draft_tree(_words(c["mask"], dev), _t(np.array(c["depth"], np.int32), dev), axes, c["pos_base"])
        self.rope = _table(c["pos_base"] + cap, c["rot"], c["theta"], dev) if not c["axes"] and c["rot"] else None
        self.out = torch.full((c["n"], c["nh"] * c["dv"]), 7.0, device=dev)
        self.ws = workspace(attn_tree_sink_workspace_bytes(self.g, c["n"], L))

    def __call__(self, stream=None):
        from mtp_speculative_draft_gb300 import attn_tree_sink
        attn_tree_sink(self.g, self.tree, self.qp, self.kp, self.vp, self.qn, self.kn, self.rope, self.sinks, self.k,
                       self.v, self.c["L"], self.out, self.ws, stream)

    def check(self, name=""):
        import torch
        from mtp_speculative_draft_gb300 import mtp_workspace_status
        torch.cuda.synchronize()
        assert mtp_workspace_status(self.ws) == 0
        c, L, n = self.c, self.c["L"], self.c["n"]
        out, k, v = _reference(c)
        got = self.out.cpu().numpy()
        assert np.isfinite(got).all()
        assert_close(got, out, name + " out", ATTN_TOL)
        kc, vc = self.k.cpu().numpy(), self.v.cpu().numpy()
        assert_close(kc[:, L:L + n], k.transpose(1, 0, 2), name + " K rows", ROPE_TOL)
        np.testing.assert_array_equal(vc[:, L:L + n], v.transpose(1, 0, 2))
        np.testing.assert_array_equal(kc[:, :L], c["kc"])
        np.testing.assert_array_equal(vc[:, :L], c["vc"])
        assert np.isnan(kc[:, L + n:]).all() and np.isnan(vc[:, L + n:]).all()


CASES = [
    dict(nh=4, nkv=2, dqk=64, dv=64, L=64, n=1),                                    # one token
    dict(nh=4, nkv=2, dqk=64, dv=64, L=0, n=1, norm=False),                         # nothing cached
    dict(nh=4, nkv=2, dqk=64, dv=64, L=0, n=5, sinks=True, tree="star"),
    dict(nh=4, nkv=2, dqk=64, dv=64, L=1, n=2),
    dict(nh=40, nkv=8, dqk=128, dv=128, L=1000, n=16, gated=True),
    dict(nh=40, nkv=8, dqk=128, dv=128, L=257, n=64, gated=True, tree="chain"),     # 320 rows a KV head
    dict(nh=16, nkv=2, dqk=256, dv=256, L=777, n=13, axes=(44, 42, 42)),
    dict(nh=16, nkv=1, dqk=256, dv=256, L=130, n=40),                               # 640 rows of one KV head
    dict(nh=32, nkv=8, dqk=192, dv=128, L=320, n=64, window=128, sinks=True, norm=False),
    dict(nh=8, nkv=4, dqk=96, dv=32, L=333, n=7, window=16, tree="chain"),
    dict(nh=8, nkv=4, dqk=64, dv=64, L=50, n=20, window=3, tree="chain", sinks=True),  # window below the tree's depth
    dict(nh=6, nkv=6, dqk=64, dv=96, L=63, n=3, window=1),                          # a row sees itself alone
    dict(nh=12, nkv=1, dqk=160, dv=224, L=515, n=11, rot=40, tree="forest"),
    dict(nh=3, nkv=3, dqk=32, dv=32, L=31, n=64, rot=10),
    dict(nh=64, nkv=1, dqk=32, dv=256, L=129, n=3, rot=0),
    dict(nh=7, nkv=1, dqk=224, dv=64, L=2000, n=9, pos_base=17),
    dict(nh=8, nkv=64 // 8, dqk=128, dv=128, L=5000, n=2),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attn_tree(dev, i):
    call = Call(_attn_case(100 + i, **CASES[i]), dev, pad=4 * (i % 3))
    call()
    call.check(str(CASES[i]))


def test_attn_tree_offsets_past_32_bits(dev):
    """The second KV head's rows start 2^31 values behind the first's."""
    import torch
    c = _attn_case(12, nh=4, nkv=2, dqk=32, dv=32, L=200, n=3)
    c["cap"] = 8
    call = Call({**c, "cap": 200 + 3}, dev)
    cap = 1 << 26
    k, v = torch.empty(2, cap, 32, device=dev), torch.empty(2, cap, 32, device=dev)
    k[:, :210], v[:, :210] = float("nan"), float("nan")
    k[:, :200], v[:, :200] = call.k[:, :200], call.v[:, :200]
    call.k, call.v = k, v
    call()
    out, kn, vn = _reference(c)
    assert_close(call.out.cpu().numpy(), out, "out", ATTN_TOL)
    assert_close(k[:, 200:203].cpu().numpy(), kn.transpose(1, 0, 2), "K rows", ROPE_TOL)
    np.testing.assert_array_equal(v[:, 200:203].cpu().numpy(), vn.transpose(1, 0, 2))
    assert torch.isnan(k[:, 203:210]).all()
    from mtp_speculative_draft_gb300 import kv_caches, kv_tree_commit
    before = k[:, 202].clone()
    kv_tree_commit(kv_caches([k], [v]), torch.tensor([2, -1, -1], dtype=torch.int32, device=dev), 200)
    assert (k[:, 200] == before).all()


def test_attn_tree_workspace_used_by_other_shapes_before(dev):
    """What an earlier call left in the workspace has no effect."""
    import torch
    a = Call(_attn_case(13, nh=16, nkv=1, dqk=256, dv=256, L=600, n=9), dev)
    b = Call(_attn_case(14, nh=5, nkv=1, dqk=96, dv=96, L=300, n=2), dev)
    b.ws = a.ws
    a.ws[1024:] = 255  # NaN everywhere behind the header
    b()
    b.check("after a fill")
    a()
    b.out.fill_(5.0)
    b()
    b.check("after another shape")
    assert torch.isfinite(b.out).all()


def test_attn_tree_repeats_bit_for_bit(dev):
    call = Call(_attn_case(1, nh=40, nkv=8, dqk=128, dv=128, L=900, n=9), dev)
    call()
    first = call.out.clone()
    for _ in range(3):
        call.out.fill_(3.0)
        call()
        assert (call.out == first).all()


def test_attn_tree_hidden_rows_have_no_effect(dev):
    """NaN and infinity in new rows that a node does not see, and in cached rows outside its window."""
    c = _attn_case(2, nh=8, nkv=2, dqk=64, dv=64, L=40, n=12, window=20, tree="star")
    for x, bad in ((c["kp"], np.nan), (c["vp"], np.inf)):
        x[5] = bad
    c["kc"][:, :21], c["vc"][:, :21] = np.nan, np.inf  # the root sees j > 20, its children j > 21
    call = Call(c, dev)
    call()
    out, _, _ = _reference(c)
    got = call.out.cpu().numpy()
    keep = [i for i in range(12) if i != 5]
    assert np.isfinite(out[keep]).all() and np.isnan(out[5]).all()
    assert_close(got[keep], out[keep], "nodes that do not see it", ATTN_TOL)
    assert np.isnan(got[5]).all()
    # a cached row that the root still sees and its children do not
    c["kc"][:, 21] = np.nan
    call = Call(c, dev)
    call()
    got = call.out.cpu().numpy()
    assert np.isnan(got[0]).all()
    keep = [i for i in range(1, 12) if i != 5]
    assert_close(got[keep], _reference(c)[0][keep], "children", ATTN_TOL)


def test_attn_tree_nan_in_a_visible_row(dev):
    c = _attn_case(3, nh=4, nkv=2, dqk=64, dv=64, L=100, n=3)
    c["kc"][1, 50, 3] = np.nan
    call = Call(c, dev)
    call()
    got = call.out.cpu().numpy().reshape(3, 4, 64)
    assert np.isnan(got[:, 2:]).all()
    assert_close(got[:, :2], _reference(c)[0].reshape(3, 4, 64)[:, :2], "other KV head", ATTN_TOL)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("L", [0, 30])
def test_attn_tree_rows_that_see_nothing(dev, L, sinks):
    c = _attn_case(4, nh=4, nkv=2, dqk=64, dv=64, L=L, n=6, window=2 if L else 0, sinks=sinks, gated=True)
    # mask bits past n are ignored
    c["mask"] = [0, 1 << 1, 0, 0xFFFF << 48, (1 << 4) | (1 << 63), 1 << 2]
    c["depth"] = [5, 5, 4, 3, 2, 5] if L else [0, 1, 0, 3, 2, 5]
    call = Call(c, dev)
    call()
    call.check()
    got = call.out.cpu().numpy()
    assert not got[0].any() and not got[3].any()


@pytest.mark.parametrize("scale", [1e-15, 1e-3, 1e3, 3e7])
def test_attn_tree_magnitudes(dev, scale):
    """Values far from 1 in V, in one K row and in single columns."""
    c = _attn_case(5, nh=8, nkv=2, dqk=128, dv=128, L=300, n=4, norm=False)
    c["vc"] *= np.float32(scale)
    c["vp"] *= np.float32(scale)
    c["vc"][:, :, 7] *= np.float32(1e-3)
    c["kc"][:, 11] *= np.float32(1e-4)
    c["kc"][:, 12] = 0
    c["qp"][1] *= np.float32(1e-6)
    call = Call(c, dev)
    call()
    got, ref = call.out.cpu().numpy().reshape(4, 8, 128), _reference(c)[0].reshape(4, 8, 128)
    small = np.arange(128) == 7
    assert_close(got[..., ~small], ref[..., ~small], "columns", ATTN_TOL)
    assert_close(got[..., small][:3], ref[..., small][:3], "small column", ATTN_TOL)


def test_attn_tree_peaked_and_large_logits(dev):
    c = _attn_case(6, nh=8, nkv=2, dqk=128, dv=128, L=500, n=4, norm=False)
    c["qp"] *= np.float32(12)
    call = Call(c, dev)
    call()
    torch_out = call.out.cpu().numpy()
    # logits up to about 60: their float32 products carry 60 / 5 times the error the tolerance is derived for
    assert_close(torch_out, _reference(c)[0], "out", 12 * ATTN_TOL)


def test_attn_tree_depth_outside_its_range(dev):
    import torch
    from mtp_speculative_draft_gb300 import mtp_workspace_status
    c = _attn_case(7, nh=4, nkv=2, dqk=64, dv=64, L=20, n=4, tree="chain")
    call = Call(c, dev)
    call.tree.tensors[1].copy_(torch.tensor([0, 1, 2, 9], dtype=torch.int32))
    call()
    torch.cuda.synchronize()
    assert mtp_workspace_status(call.ws) == 5
    assert_close(call.out.cpu().numpy(), _reference(c)[0], "nearest depth", ATTN_TOL)  # 9 counts as 3


def test_attn_tree_chain_matches_decode_attention(dev):
    """A chain is what attn_decode_sink computes for consecutive rows."""
    import torch
    from mtp_speculative_draft_gb300 import attn_decode_sink
    call = Call(_attn_case(8, nh=8, nkv=2, dqk=128, dv=128, L=70, n=4, tree="chain", gated=True), dev)
    call()
    c = call.c
    out, k, v = torch.zeros_like(call.out), call.k.clone(), call.v.clone()
    attn_decode_sink(call.g, call.qp, call.kp, call.vp, call.qn, call.kn, call.rope, None, k, v, 70, c["cap"], 4, out)
    assert_close(call.out.cpu().numpy(), out.cpu().numpy(), "decode", 2 * ATTN_TOL)
    assert_close(call.k[:, 70:74].cpu().numpy(), k[:, 70:74].cpu().numpy(), "K rows", 2 * ROPE_TOL)


def test_attn_tree_graphs_streams_and_a_shared_workspace(dev):
    """Two captured graphs on one workspace, replayed on another stream than the capture's."""
    import torch
    a = Call(_attn_case(9, nh=8, nkv=2, dqk=128, dv=128, L=600, n=5), dev)
    b = Call(_attn_case(10, nh=40, nkv=8, dqk=128, dv=128, L=90, n=30), dev)
    ws = max(a.ws, b.ws, key=lambda t: t.numel())
    a.ws = b.ws = ws
    a()
    b()
    torch.cuda.synchronize()
    graphs = []
    for call in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    side = torch.cuda.Stream()
    a.out.zero_()
    b.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(4):
            graphs[0].replay()
            graphs[1].replay()
    side.synchronize()
    a.check("first graph")
    b.check("second graph")


def test_wrappers_refuse_what_the_kernels_cannot_read(dev):
    """Broadcast rows, wrong types, short or non-contiguous tensors: refused before any launch."""
    import torch
    import mtp_speculative_draft_gb300 as M
    call = Call(_attn_case(11, nh=4, nkv=2, dqk=64, dv=64, L=10, n=3), dev)
    good = dict(qp=call.qp, kp=call.kp, out=call.out, k=call.k)
    for name, bad, error in (
            ("qp", call.qp[:1].expand(3, -1), ValueError),      # one row seen three times
            ("qp", call.qp.double(), TypeError), ("qp", call.qp[:, ::2], ValueError),
            ("kp", call.kp[:2], ValueError), ("kp", call.kp.cpu(), ValueError),
            ("out", call.out[:2], ValueError), ("out", call.out.t(), ValueError), ("out", call.out.half(), TypeError),
            ("k", call.k[:1], ValueError)):
        for key, value in {**good, name: bad}.items():
            setattr(call, key, value)
        with pytest.raises(error):
            call()
    for key, value in good.items():
        setattr(call, key, value)
    call()
    call.check()
    x = torch.zeros(1, 100, device=dev)
    tok, val = torch.zeros(4, dtype=torch.int32, device=dev), torch.zeros(4, device=dev)
    with pytest.raises(ValueError):
        M.logit_rules_argmax(M.logit_rules(100), x.expand(4, 100), tok, val)
    with pytest.raises(ValueError):  # the mask has fewer rows than the logits
        M.logit_rules_argmax(M.logit_rules(100, allow=torch.zeros(3, 4, dtype=torch.int32, device=dev)),
                             torch.zeros(4, 100, device=dev), tok, val)
    with pytest.raises(ValueError):  # one cache twice
        M.kv_caches([call.k, call.k], [call.v, call.v.clone()])
    with pytest.raises(M._lib.MtpError):  # rows that overlap
        ax = M.rope_axes((16,), torch.zeros(1, 4, dtype=torch.int32, device=dev), torch.zeros(64, device=dev))
        M.rope_axes_rows(ax, [(torch.zeros(1, 2, 32, device=dev).expand(4, 2, 32), torch.zeros(4, 2, 32, device=dev), None)])


def test_attn_tree_two_streams_at_once(dev):
    """Calls with workspaces of their own on two streams at the same time."""
    import torch
    calls = [Call(_attn_case(15, nh=40, nkv=8, dqk=128, dv=128, L=3000, n=40), dev),
             Call(_attn_case(16, nh=16, nkv=2, dqk=256, dv=256, L=2500, n=20, sinks=True), dev)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for call, stream in zip(calls, streams):
            call(stream)
    for call in calls:
        call.check()


def test_captured_calls_follow_their_tensors(dev):
    """A replayed graph reads the tree, the rules' tables and the positions of the replay."""
    import torch
    import mtp_speculative_draft_gb300 as M
    c = _attn_case(17, nh=8, nkv=2, dqk=64, dv=64, L=70, n=20, axes=(12, 10, 10))
    call = Call(c, dev)
    mask, depth, axes = call.tree.tensors
    rules = _rules_case(3, 20, 3000, n_path=20, n_bias=5, allow="rows")
    r = _rules_device(rules, dev)
    logits, out = _t(rules["logits"], dev), torch.zeros(20, 3000, device=dev)
    tok, val = torch.zeros(20, dtype=torch.int32, device=dev), torch.zeros(20, device=dev)
    ws = M.workspace(M.logit_rules_argmax_workspace_bytes(20))
    call()
    M.logit_rules_argmax(r, logits, tok, val, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        M.logit_rules_argmax(r, logits, tok, val, out, ws)
    for seed, kind in ((18, "chain"), (19, "star"), (20, "forest")):
        n = _attn_case(seed, nh=8, nkv=2, dqk=64, dv=64, L=70, n=20, axes=(12, 10, 10), tree=kind)
        mask.copy_(_words(n["mask"], dev))
        depth.copy_(_t(np.array(n["depth"], np.int32), dev))
        axes.tensors[0].copy_(_t(n["pos"], dev))
        for x, y in ((call.qp, n["qp"]), (call.kp, n["kp"]), (call.vp, n["vp"]), (call.k[:, :70], n["kc"]),
                     (call.v[:, :70], n["vc"]), (call.qn, n["qn"]), (call.kn, n["kn"])):
            x.copy_(_t(y, dev))
        call.c = n
        new = _rules_case(seed, 20, 3000, n_path=20, n_bias=5, allow="rows")
        counts, btok, b, allow, ptok, pmask = r.tensors
        for x, y in ((counts, np.asarray(new["counts"]).astype(np.uint32).view(np.int32)), (btok, new["bias_tokens"]),
                     (b, new["bias"]), (allow, new["allow"].view(np.int32)), (ptok, new["path_tokens"]), (logits, new["logits"])):
            x.copy_(_t(y, dev))
        pmask.copy_(_words(new["path_mask"], dev))
        g.replay()
        call.check(kind)
        np.testing.assert_array_equal(out.cpu().numpy(), _rules_reference(new))
        assert tok.tolist() == [t for t, _ in T.greedy(_rules_reference(new))]


# ------------------------------------------------------------------ logit rules
def _rules_case(seed, rows, V, n_path=0, n_bias=0, allow=None, counts=True, rep=1.3, freq=0.4, pres=0.3):
    rng = np.random.default_rng(seed)
    c = dict(logits=(3 * rng.standard_normal((rows, V))).astype(np.float32), rep=rep, freq=freq, pres=pres)
    c["counts"] = (rng.integers(0, 5, V) * (rng.random(V) < 0.2)).astype(np.int64) if counts else None
    if counts:
        c["counts"] |= np.where(rng.random(V) < 0.1, 1 << 31, 0)
    c["bias_tokens"] = rng.integers(0, V, n_bias).astype(np.int32)  # tokens repeat in small vocabularies
    c["bias"] = rng.standard_normal(n_bias).astype(np.float32)
    c["path_tokens"] = rng.integers(0, V, n_path).astype(np.int32)
    c["path_mask"] = [int(w) for w in rng.integers(0, 1 << 63, rows, dtype=np.uint64) * np.uint64(2) + np.uint64(1)]
    words = (V + 31) // 32
    shape = {None: None, "rows": (rows, words + 2), "one": (words,)}[allow]
    c["allow"] = rng.integers(0, 1 << 32, shape, dtype=np.uint64).astype(np.uint32) if shape else None
    return c


def _rules_device(c, dev):
    from mtp_speculative_draft_gb300 import logit_rules
    i32 = lambda a: None if a is None else _t(np.asarray(a).astype(np.uint32).view(np.int32), dev)  # noqa: E731
    nb, npath = len(c["bias"]), len(c["path_tokens"])
    return logit_rules(c["logits"].shape[1], c["rep"], c["freq"], c["pres"], i32(c["counts"]),
                       _t(c["bias_tokens"], dev) if nb else None, _t(c["bias"], dev) if nb else None, i32(c["allow"]),
                       _t(c["path_tokens"], dev) if npath else None, _words(c["path_mask"], dev) if npath else None)


def _rules_reference(c, dtype=np.float32):
    return T.logit_rules(c["logits"], c["counts"], c["rep"], c["freq"], c["pres"], list(zip(c["bias_tokens"], c["bias"])),
                         c["allow"], c["path_tokens"], c["path_mask"], dtype)


@pytest.mark.parametrize("rows,V,kw", [
    (1, 1, dict(counts=False)),
    (1, 4096, dict(n_bias=4, allow="rows")),
    (2, 33, dict(n_bias=70, n_path=64, allow="one")),          # every token many times
    (3, 2047, dict(n_path=7, allow="rows")),
    (5, 2049, dict(n_bias=33, n_path=64)),
    (16, 10007, dict(n_bias=300, n_path=16, allow="rows")),
    (64, 5001, dict(n_path=64, allow="rows", rep=0.7, freq=-0.2)),
    (1, 151936, dict(n_bias=1000, allow="rows")),
    (130, 300, dict(counts=False, n_bias=1, rep=1.0, freq=0.0, pres=0.0)),
    (9, 70000, dict(counts=False, n_path=64)),                 # the path alone counts
    (2, 500, dict(n_bias=700, n_path=3)),                      # more bias entries in a chunk than it keeps at hand
    (70, 4097, dict(n_bias=9, n_path=64, allow="one")),        # several rows a CTA where chunks are few
])
@pytest.mark.parametrize("out", ["none", "new", "in place"])
def test_logit_rules(dev, rows, V, kw, out):
    import torch
    from mtp_speculative_draft_gb300 import logit_rules_argmax
    c = _rules_case(rows + V, rows, V, **kw)
    pad = 5 if out == "new" else 0
    x = _t(np.pad(c["logits"], ((0, 0), (0, pad)), constant_values=np.nan), dev)[:, :V]
    y = {"none": None, "new": torch.full((rows, V + 3), 7.0, device=dev)[:, :V], "in place": x}[out]
    tok, val = torch.full((rows,), 9, dtype=torch.int32, device=dev), torch.zeros(rows, device=dev)
    rules = _rules_device(c, dev)
    ws = logit_rules_argmax(rules, x, tok, val, y)
    ref = _rules_reference(c)
    want = T.greedy(ref)
    assert tok.tolist() == [t for t, _ in want]
    assert val.tolist() == [v for _, v in want]
    if y is not None:
        np.testing.assert_array_equal(y.cpu().numpy(), ref)
        exact = _rules_reference(c, np.float64)
        fin = np.isfinite(exact)
        # four roundings of values no larger than theta * |l| + the penalties and biases
        assert np.abs(ref[fin] - exact[fin]).max() <= 4 * 2.0 ** -24 * 4 * np.abs(c["logits"]).max() + 1e-6 * max(1, len(c["bias"]))
    if out == "new":
        assert (y._base[:, V:] == 7.0).all()  # columns past the vocabulary stay
    if out != "in place":  # the workspace is clean again
        logit_rules_argmax(rules, x, tok.zero_(), val, y, ws)
        assert tok.tolist() == [t for t, _ in want]


def test_logit_rules_ties_infinities_and_empty_rows(dev):
    import torch
    from mtp_speculative_draft_gb300 import logit_rules, logit_rules_argmax
    V = 5000
    x = torch.full((6, V), -1.0, device=dev)
    x[0, 4999] = x[0, 2500] = 3.0                        # ties: the lowest index
    x[1, 17], x[1, 3] = float("nan"), float("inf")       # NaN never wins
    x[2] = float("-inf")                                 # nothing above -inf
    x[3] = float("nan")
    x[4, 100], x[4, 40] = 0.0, -0.0                      # zeros are equal
    x[4, 200] = 0.0
    x[5] = 5.0                                           # all forbidden
    allow = torch.full((6, (V + 31) // 32), -1, dtype=torch.int32, device=dev)
    allow[5] = 0
    tok, val = torch.zeros(6, dtype=torch.int32, device=dev), torch.zeros(6, device=dev)
    logit_rules_argmax(logit_rules(V, allow=allow), x, tok, val)
    assert tok.tolist() == [2500, 3, -1, -1, 40, -1]
    assert val.tolist() == [3.0, float("inf"), float("-inf"), float("-inf"), 0.0, float("-inf")]


def test_token_counts(dev):
    import torch
    from mtp_speculative_draft_gb300 import mtp_token_counts, mtp_workspace_status, workspace
    ws = workspace(1024)
    counts = torch.zeros(1000, dtype=torch.int32, device=dev)
    rng = np.random.default_rng(3)
    a, b = rng.integers(0, 50, 3000).astype(np.int32), rng.integers(0, 1000, 300).astype(np.int32)
    a[::7] = -1
    mtp_token_counts(counts, _t(a, dev), False, ws)
    mtp_token_counts(counts, _t(b, dev), True, ws)
    want = np.bincount(a[a >= 0], minlength=1000)
    want[b] |= 1 << 31
    np.testing.assert_array_equal(counts.cpu().numpy().view(np.uint32), want)
    assert mtp_workspace_status(ws) == 0
    mtp_token_counts(counts, torch.tensor([5, 1000], dtype=torch.int32, device=dev), False, ws)
    assert mtp_workspace_status(ws) == 2
    assert int(counts[5]) & 0x7FFFFFFF == want[5] % (1 << 31) + 1


# ------------------------------------------------------------------ plan, accept, commit
@pytest.mark.parametrize("n,kind", [(1, "random"), (2, "chain"), (33, "star"), (64, "chain"), (64, "random"), (40, "forest")])
def test_tree_plan(dev, n, kind):
    import torch
    from mtp_speculative_draft_gb300 import mtp_tree_plan, mtp_workspace_status
    parents = _parents(np.random.default_rng(n), n, kind)
    mask, depth = torch.zeros(n, dtype=torch.int64, device=dev), torch.zeros(n, dtype=torch.int32, device=dev)
    ws = mtp_tree_plan(_t(np.array(parents, np.int32), dev), mask, depth)
    m, d = T.tree_plan(parents)
    assert mask.cpu().numpy().view(np.uint64).tolist() == m and depth.tolist() == d
    assert mtp_workspace_status(ws) == 0


def test_tree_plan_bad_parents(dev):
    import torch
    from mtp_speculative_draft_gb300 import mtp_tree_plan, mtp_workspace_status
    mask, depth = torch.zeros(5, dtype=torch.int64, device=dev), torch.zeros(5, dtype=torch.int32, device=dev)
    ws = mtp_tree_plan(torch.tensor([-1, 1, 0, 9, -7], dtype=torch.int32, device=dev), mask, depth)
    assert mask.tolist() == [1, 2, 5, 8, 16] and depth.tolist() == [0, 0, 1, 0, 0]  # they count as roots
    assert mtp_workspace_status(ws) == 5


@pytest.mark.parametrize("seed", range(12))
def test_tree_accept_and_commit(dev, seed):
    import torch
    from mtp_speculative_draft_gb300 import kv_caches, kv_tree_commit, mtp_tree_accept, mtp_workspace_status
    rng = np.random.default_rng(seed)
    n = [1, 2, 5, 16, 33, 64][seed % 6]
    layers, nkv, dqk, dv, L = [(1, 2, 64, 64, 7), (3, 1, 256, 32, 0), (70, 3, 4, 12, 5)][seed % 3]
    parents = _parents(rng, n, ["random", "chain", "star", "forest"][seed % 4])
    tokens = rng.integers(0, 4, n)  # siblings share tokens
    verify = rng.integers(0, 4, n)
    if seed % 2:
        for i in range(n):  # long paths
            kids = [j for j in range(n) if parents[j] == i]
            if kids:
                verify[i] = tokens[kids[rng.integers(len(kids))]]
    i32 = lambda a: _t(np.array(a, np.int32), dev)  # noqa: E731
    path, emitted, count = i32([9] * n), i32([9] * n), i32([0])
    mtp_tree_accept(i32(parents), i32(tokens), i32(verify), path, emitted, count)
    want, em = T.tree_accept(parents, tokens, verify)
    assert path.tolist() == want + [-1] * (n - len(want))
    assert emitted.tolist() == em + [-1] * (n - len(want)) and count.item() == len(want)
    cap = L + n + 3
    ks = [torch.randn(nkv, cap, dqk, device=dev) for _ in range(layers)]
    vs = [torch.randn(nkv, cap, dv, device=dev) for _ in range(layers)]
    before = [(k.clone(), v.clone()) for k, v in zip(ks, vs)]
    ws = kv_tree_commit(kv_caches(ks, vs), path, L)
    assert mtp_workspace_status(ws) == 0
    for l in range(layers):
        for x, b in zip((ks[l], vs[l]), before[l]):
            ref = b.clone()
            for j, p in enumerate(want):
                ref[:, L + j] = b[:, L + p]
            assert (x == ref).all()


def test_commit_of_a_bad_path(dev):
    import torch
    from mtp_speculative_draft_gb300 import kv_caches, kv_tree_commit, mtp_workspace_status
    k, v = torch.randn(2, 20, 32, device=dev), torch.randn(2, 20, 32, device=dev)
    k0 = k.clone()
    for path, moved in (([0, 3, 1, 2], 2), ([1, 4, 2, 3], 1), ([2, -1, 3, 3], 1)):
        k.copy_(k0)
        ws = kv_tree_commit(kv_caches([k], [v]), torch.tensor(path, dtype=torch.int32, device=dev), 6)
        ref = k0.clone()
        for j in range(moved):
            ref[:, 6 + j] = k0[:, 6 + path[j]]
        assert (k == ref).all()
        assert mtp_workspace_status(ws) == (5 if -1 not in path else 0)


def test_round_of_a_tree(dev):
    """Plan, attention of two layers, head, rules, accept, count update and commit as one captured round,
    then the accepted rows serve as the cache of a second attention."""
    import torch
    import mtp_speculative_draft_gb300 as M
    rng = np.random.default_rng(77)
    n, nh, nkv, d, L, V = 12, 8, 2, 64, 90, 2000
    parents = _parents(rng, n, "random")
    cases = [_attn_case(s, nh=nh, nkv=nkv, dqk=d, dv=d, L=L, n=n) for s in (20, 21)]
    for c in cases:
        c["parents"] = parents
        c["mask"], c["depth"] = T.tree_plan(parents)
    calls = [Call(c, dev) for c in cases]
    i32 = lambda a: _t(np.array(a, np.int32), dev)  # noqa: E731
    par, mask, depth = i32(parents), torch.zeros(n, dtype=torch.int64, device=dev), torch.zeros(n, dtype=torch.int32, device=dev)
    for c in calls:
        c.tree = M.draft_tree(mask, depth)
    tokens = rng.integers(0, V, n)
    logits = rng.standard_normal((n, V)).astype(np.float32)
    counts = np.zeros(V, np.int64)
    counts[rng.integers(0, V, 200)] += 2
    for i in range(n):  # the verifier favours one child of each node, before penalties
        kids = [j for j in range(n) if parents[j] == i]
        if kids:
            logits[i, tokens[kids[0]]] = 9.0
    tl, tc, tt = _t(logits, dev), i32(counts), i32(tokens)
    rules = M.logit_rules(V, 1.2, 0.1, 0.2, tc, path_tokens=tt, path_mask=mask)
    pick, val = torch.zeros(n, dtype=torch.int32, device=dev), torch.zeros(n, device=dev)
    path, emitted, count = (torch.zeros(k, dtype=torch.int32, device=dev) for k in (n, n, 1))
    ws, rws = M.workspace(1024), M.workspace(M.logit_rules_argmax_workspace_bytes(n))
    caches = M.kv_caches([c.k for c in calls], [c.v for c in calls])

    def round_():
        M.mtp_tree_plan(par, mask, depth, ws)
        for c in calls:
            c()
        M.logit_rules_argmax(rules, tl, pick, val, None, rws)
        M.mtp_tree_accept(par, tt, pick, path, emitted, count)
        M.mtp_token_counts(tc, emitted, False, ws)
        M.kv_tree_commit(caches, path, L, ws)

    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        round_()
    tc.copy_(i32(counts))
    g.replay()
    torch.cuda.synchronize()
    mk, dp = T.tree_plan(parents)
    ref = T.logit_rules(logits, counts, 1.2, 0.1, 0.2, path_tokens=tokens, path_mask=mk, dtype=np.float32)
    want, em = T.tree_accept(parents, tokens, [t for t, _ in T.greedy(ref)])
    assert len(want) > 1 and path.tolist()[:len(want)] == want and count.item() == len(want)
    np.testing.assert_array_equal(tc.cpu().numpy(), counts + np.bincount(em, minlength=V))
    for c in calls:
        out, k, v = _reference(c.c)
        assert_close(c.out.cpu().numpy(), out, "tree rows", ATTN_TOL)
        a = len(want)
        assert_close(c.k[:, L:L + a].cpu().numpy(), k[want].transpose(1, 0, 2), "kept K rows", ROPE_TOL)
        # the next token attends to the kept rows as to any cached ones
        nxt = _attn_case(30, nh=nh, nkv=nkv, dqk=d, dv=d, L=L + a, n=1)
        nxt["kc"], nxt["vc"] = (np.concatenate([c.c[x], y[want].transpose(1, 0, 2)], 1) for x, y in (("kc", k), ("vc", v)))
        follow = Call(nxt, dev)
        follow.k[:, :L + a].copy_(c.k[:, :L + a])
        follow()
        assert_close(follow.out.cpu().numpy(), _reference(nxt)[0], "next token", ATTN_TOL)
