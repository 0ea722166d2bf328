"""The beam search's step on the GPU against the float64 reference.

Tolerances:

* attention, errors scaled by max(|ref|, rms(ref)): as derived for the tree's rows (test_gpu_tree.py), whose
  operands, sums and rotations these are; keys of a tail are read as float32, which is less than that.
* selection: a term of the sum of exponentials is off by 2 units of exp2 and the rounding of its argument
  (2^-22 in all at most), 32 of them are added in float32 (8 roundings a term at most: 2^-21), the rest in 64
  bits: a normaliser, and so a score, is off by 2^-20.4 at most before its own rounding (half a step).  Two
  candidates of different beams may change places when their scores differ by less than twice that; tokens of one
  beam, and equal scores of equal beams, may not.
* tails: bit for bit.
"""

import math

import numpy as np
import pytest

from helpers import assert_close
from oracle import beam_oracle as B
from oracle import tree_oracle as T
from test_gpu_tree import ATTN_TOL, ROPE_TOL, _t, _table, dev  # noqa: F401

pytestmark = pytest.mark.gpu

SUM_TOL = 2.0 ** -20.4


# ------------------------------------------------------------------ attn_prefix_sink
def _attn_case(seed, nh, nkv, dqk, dv, plen, tlen, m=1, rot=None, window=0, gated=False, norm=True, sinks=False, axes=None,
               pos_base=0, loose=(0, 0)):
    """``plen``, ``tlen``: rows of prompts and tails; ``loose``: how far the call's bounds lie above them."""
    rng = np.random.default_rng(seed)
    rot = dqk if rot is None else rot
    groups, seqs = len(plen), len(tlen)
    c = dict(nh=nh, nkv=nkv, dqk=dqk, dv=dv, plen=plen, tlen=tlen, m=m, rot=rot, window=window, gated=gated, axes=axes,
             pos_base=pos_base, theta=1e4, pmax=max(plen) + loose[0], tmax=max(0, *tlen) + loose[1])
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    rows = seqs * m
    c["qp"], c["kp"], c["vp"] = f(rows, nh * dqk * (2 if gated else 1)), f(rows, nkv * dqk), f(rows, nkv * dv)
    # rows behind a length hold NaN and take no part
    cut = lambda x, n: np.where((np.arange(x.shape[2]) < np.array(n)[:, None])[:, None, :, None], x, np.float32(np.nan))  # noqa: E731
    c["kpre"], c["vpre"] = cut(f(groups, nkv, c["pmax"] + 2, dqk), plen), cut(f(groups, nkv, c["pmax"] + 2, dv), plen)
    tcap = c["tmax"] + m + 3
    c["kt"], c["vt"] = cut(f(seqs, nkv, tcap, dqk), tlen), cut(f(seqs, nkv, tcap, dv), tlen)
    c["qn"], c["kn"] = (1 + 0.1 * f(dqk), 1 + 0.1 * f(dqk)) if norm else (None, None)
    c["sinks"] = f(nh) if sinks else None
    c["pos"] = rng.integers(0, 300, (len(axes), rows)).astype(np.int32) if axes else None
    return c


def _reference(c):
    nh, nkv, dqk, dv, m = (c[k] for k in ("nh", "nkv", "dqk", "dv", "m"))
    rows, seqs, per = len(c["tlen"]) * m, len(c["tlen"]), len(c["tlen"]) // len(c["plen"])
    raw = c["qp"].reshape(rows, nh, -1)
    sec = c["axes"] or (c["rot"] // 2,)
    pos = c["pos"] if c["axes"] else [[c["pos_base"] + c["plen"][b // per] + max(0, c["tlen"][b]) + i
                                       for b in range(seqs) for i in range(m)]]
    turn = (lambda x: T.rope_axes(x, pos, sec, True, c["theta"])) if c["rot"] else (lambda x: np.asarray(x, np.float64))
    q = turn(T.head_norm(raw[..., :dqk], c["qn"], 1e-6))
    k = turn(T.head_norm(c["kp"].reshape(rows, nkv, dqk), c["kn"], 1e-6))
    v = c["vp"].reshape(rows, nkv, dv)
    out = B.prefix_attention(q, k, v, c["kpre"], c["vpre"], c["kt"], c["vt"], c["plen"], c["tlen"], m, c["window"],
                             c["sinks"], raw[..., dqk:] if c["gated"] else None)
    return out, k, v


class Call:
    """Device copies of a case's inputs and its call."""

    def __init__(self, c, dev, pad=0):  # noqa: F811
        import torch
        import mtp_speculative_draft_gb300 as M
        self.c, nkv = c, c["nkv"]
        strided = lambda a: _t(np.pad(a, ((0, 0), (0, pad)), constant_values=np.nan), dev)[:, :a.shape[1]]  # noqa: E731
        self.qp, self.kp, self.vp = strided(c["qp"]), strided(c["kp"]), strided(c["vp"])
        self.kpre, self.vpre, self.kt, self.vt = (_t(c[n], dev) for n in ("kpre", "vpre", "kt", "vt"))
        self.qn, self.kn, self.sinks = _t(c["qn"], dev), _t(c["kn"], dev), _t(c["sinks"], dev)
        self.g = M.attn_geom(c["nh"], nkv, c["dqk"], c["dv"], c["rot"], c["window"], c["gated"])
        axes = None
        if c["axes"]:
            axes = M.rope_axes(c["axes"], _t(c["pos"], dev), _table(300, c["rot"], c["theta"], dev), interleaved=True)
        self.plen, self.tlen = (_t(np.array(c[n], np.int32), dev) for n in ("plen", "tlen"))
        self.batch = M.prefix_batch(self.plen, self.tlen, c["pmax"], c["tmax"], c["m"], axes, c["pos_base"])
        top = c["pos_base"] + c["pmax"] + c["tmax"] + c["m"]
        self.rope = _table(top, c["rot"], c["theta"], dev) if not c["axes"] and c["rot"] else None
        self.out = torch.full((len(c["tlen"]) * c["m"], c["nh"] * c["dv"]), 7.0, device=dev)
        self.ws = M.workspace(M.attn_prefix_sink_workspace_bytes(self.g, self.batch))

    def __call__(self, stream=None):
        import mtp_speculative_draft_gb300 as M
        M.attn_prefix_sink(self.g, self.batch, self.qp, self.kp, self.vp, self.qn, self.kn, self.rope, self.sinks, self.kpre,
                           self.vpre, self.kt, self.vt, self.out, self.ws, stream)

    def check(self, name="", tol=ATTN_TOL):
        import torch
        import mtp_speculative_draft_gb300 as M
        torch.cuda.synchronize()
        assert M.mtp_workspace_status(self.ws) == 0
        c, m = self.c, self.c["m"]
        out, k, v = _reference(c)
        got = self.out.cpu().numpy().reshape(-1, c["nh"], c["dv"])
        kt, vt = self.kt.cpu().numpy(), self.vt.cpu().numpy()
        for b, t in enumerate(c["tlen"]):
            rows = slice(b * m, b * m + m)
            keep = np.ones(kt.shape[2], bool)
            if t < 0:
                assert (got[rows] == 7).all()
            else:
                keep[t:t + m] = False
                assert_close(got[rows], np.array(out[rows]), f"{name} out of sequence {b}", tol)
                assert_close(kt[b, :, t:t + m], k[rows].transpose(1, 0, 2), name + " K rows", ROPE_TOL)
                np.testing.assert_array_equal(vt[b, :, t:t + m], v[rows].transpose(1, 0, 2))
            np.testing.assert_array_equal(kt[b][:, keep], c["kt"][b][:, keep])
            np.testing.assert_array_equal(vt[b][:, keep], c["vt"][b][:, keep])


CASES = [
    dict(nh=4, nkv=2, dqk=64, dv=64, plen=[64], tlen=[3] * 4),                                 # the tail launch alone
    dict(nh=1, nkv=1, dqk=32, dv=32, plen=[0], tlen=[0]),                                      # a row that sees itself alone
    dict(nh=4, nkv=2, dqk=64, dv=64, plen=[1], tlen=[0, 1, -1], norm=False),
    dict(nh=4, nkv=4, dqk=64, dv=64, plen=[65], tlen=[0]),                                     # one sequence, one split
    dict(nh=6, nkv=2, dqk=96, dv=96, plen=[200, 0, 77], tlen=[5, -1, 9, 0, 64, 7]),            # an empty prompt among others
    dict(nh=40, nkv=8, dqk=128, dv=128, plen=[1000], tlen=[17] * 8, gated=True),
    dict(nh=40, nkv=8, dqk=128, dv=128, plen=[300], tlen=[(7 * i) % 40 for i in range(70)], gated=True),  # 350 rows a KV head
    dict(nh=16, nkv=2, dqk=256, dv=256, plen=[513, 300], tlen=[40, 0, 31, 129, -1, 8], axes=(44, 42, 42)),
    dict(nh=32, nkv=8, dqk=192, dv=128, plen=[320], tlen=[77, 3, 200, 0, 128], m=4, window=128, norm=False, sinks=True),
    dict(nh=8, nkv=4, dqk=96, dv=32, plen=[333], tlen=[0, 2, 30], m=7, window=16),             # the edge is most of the window
    dict(nh=8, nkv=4, dqk=64, dv=64, plen=[500, 80], tlen=[30, 1, 0, 200], window=100, sinks=True),
    dict(nh=6, nkv=6, dqk=64, dv=96, plen=[90], tlen=[3, 0], m=5, window=1, sinks=True),       # rows see themselves alone
    dict(nh=6, nkv=6, dqk=64, dv=96, plen=[900], tlen=[3, 0], m=16, window=9),                 # a window below the new rows
    dict(nh=12, nkv=1, dqk=160, dv=224, plen=[515], tlen=[11, 12, 700], rot=40),
    dict(nh=3, nkv=3, dqk=32, dv=32, plen=[131], tlen=[31] * 64, rot=10),
    dict(nh=64, nkv=1, dqk=32, dv=256, plen=[129], tlen=[3, 90, 1], rot=0),
    dict(nh=128, nkv=2, dqk=32, dv=64, plen=[100], tlen=[300, 2], m=3),                        # 64 heads a KV head
    dict(nh=7, nkv=1, dqk=224, dv=64, plen=[2000], tlen=[9], pos_base=17),
    dict(nh=8, nkv=8, dqk=128, dv=128, plen=[5000], tlen=[0, 1], loose=(300, 40)),
    dict(nh=8, nkv=8, dqk=128, dv=128, plen=[70], tlen=[3000, 2999], m=2),                     # tails over clusters
    dict(nh=2, nkv=1, dqk=256, dv=128, plen=[70], tlen=[1500]),
    dict(nh=5, nkv=1, dqk=128, dv=256, plen=[0], tlen=[1100, 9], sinks=True, loose=(0, 500)),
    dict(nh=4, nkv=1, dqk=64, dv=64, plen=[400] * 5, tlen=[7] * 5, loose=(1, 0)),              # a sequence a prompt
    dict(nh=2, nkv=2, dqk=64, dv=64, plen=[100], tlen=[-1, -1, -1]),                           # no sequence at all
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(dev, i):  # noqa: F811
    call = Call(_attn_case(500 + i, **CASES[i]), dev, pad=4 * (i % 3))
    call()
    call.check(str(CASES[i]))


def test_attention_of_tails_below_an_empty_prompt_array(dev):  # noqa: F811
    """prefix_max 0: no arrays of prompts at all."""
    c = _attn_case(1, nh=8, nkv=2, dqk=64, dv=64, plen=[0], tlen=[90, 0, 5])
    call = Call(c, dev)
    call.kpre = call.vpre = None
    call()
    call.check()


def test_one_sequence_is_decode_attention(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    call = Call(_attn_case(2, nh=8, nkv=2, dqk=128, dv=128, plen=[0], tlen=[70], m=4, gated=True), dev)
    k, v, out = call.kt[0].clone(), call.vt[0].clone(), torch.zeros_like(call.out)
    call()
    M.attn_decode_sink(call.g, call.qp, call.kp, call.vp, call.qn, call.kn, call.rope, None, k, v, 70, k.shape[1], 4, out)
    assert_close(call.out.cpu().numpy(), out.cpu().numpy(), "decode", 2 * ATTN_TOL)
    assert_close(call.kt[0, :, 70:74].cpu().numpy(), k[:, 70:74].cpu().numpy(), "K rows", 2 * ROPE_TOL)


@pytest.mark.parametrize("where", ["prompt", "tail"])
def test_attention_offsets_past_32_bits(dev, where):  # noqa: F811
    """The second KV head's rows (of the first sequence) start 2^31 values behind the first's."""
    import torch
    c = _attn_case(12, nh=4, nkv=2, dqk=32, dv=32, plen=[200], tlen=[90])
    call = Call(c, dev)
    cap = 1 << 26
    for name in ("kpre", "vpre") if where == "prompt" else ("kt", "vt"):
        big, small = torch.empty(1, 2, cap, 32, device=dev), getattr(call, name)
        big[:, :, :small.shape[2]] = small
        setattr(call, name, big)
    call()
    torch.cuda.synchronize()
    if where == "tail":
        call.kt, call.vt = call.kt[:, :, :c["kt"].shape[2]].clone(), call.vt[:, :, :c["vt"].shape[2]].clone()
    call.check()


def test_attention_of_many_sequences(dev):  # noqa: F811
    """1024 sequences: lengths and rows of all of them."""
    c = _attn_case(13, nh=2, nkv=1, dqk=32, dv=32, plen=[100, 90], tlen=[i % 23 - 1 for i in range(1024)], window=60)
    call = Call(c, dev)
    call()
    call.check()


def test_workspace_used_by_other_calls_before(dev):  # noqa: F811
    """What an earlier call of any kind left in the workspace has no effect, and its other users' state stays."""
    import torch
    import mtp_speculative_draft_gb300 as M
    a = Call(_attn_case(14, nh=16, nkv=1, dqk=256, dv=256, plen=[600], tlen=[9, 30, 2]), dev)
    b = Call(_attn_case(15, nh=5, nkv=1, dqk=96, dv=96, plen=[300], tlen=[2]), dev)
    x = np.random.default_rng(4).standard_normal((64, 9001)).astype(np.float32)
    logits, want = _t(x, dev), [t for t, _ in T.greedy(x)]
    tok, val = torch.empty(64, dtype=torch.int32, device=dev), torch.empty(64, device=dev)
    score = torch.zeros(64, device=dev)
    out = [torch.empty(8, 8, dtype=d, device=dev) for d in (torch.int32, torch.int32, torch.float32)]
    beams = M.beam_set(8, 8, 9001, score)
    ref = B.beam_select(x, 8, 8, 8, np.zeros(64))
    ws = M.workspace(max(a.ws.numel(), b.ws.numel(), M.logit_rules_argmax_workspace_bytes(64),
                         M.beam_select_workspace_bytes(beams, 8)))
    a.ws = b.ws = ws
    ws[1024 + 16384:] = 255  # NaN behind the header and the rules' joins
    for _ in range(2):
        for call in (a, b):
            call.kt.copy_(_t(call.c["kt"], dev))
            call.out.fill_(7.0)
            call()
            call.check()
            M.logit_rules_argmax(M.logit_rules(9001), logits, tok, val, None, ws)
            assert tok.tolist() == want
            M.beam_select(beams, logits, 8, *out, ws=ws)
            assert out[1].tolist() == ref[1].tolist()


def test_attention_repeats_bit_for_bit(dev):  # noqa: F811
    call = Call(_attn_case(16, nh=40, nkv=8, dqk=128, dv=128, plen=[900], tlen=[40, 700, 3]), dev)
    call()
    first = call.out.clone()
    for _ in range(3):
        call.out.fill_(3.0)
        call()
        assert (call.out == first).all()


def test_hidden_rows_have_no_effect(dev):  # noqa: F811
    """NaN and infinity in new rows behind a row, in rows outside its window and in other sequences."""
    c = _attn_case(17, nh=8, nkv=2, dqk=64, dv=64, plen=[200, 300], tlen=[40, 0, 10, 120], m=3, window=100)
    lo = 200 + 0 + 1 - 100                                  # the first prompt's row that sequence 1's row 0 still sees
    c["kpre"][0, :, :lo], c["vpre"][0, :, :lo] = np.nan, np.inf
    c["kt"][3, :, :21], c["vt"][3, :, :21] = np.inf, np.nan  # row 0 of sequence 3 sees tail rows above 20
    c["kp"][2], c["vp"][2] = np.nan, np.inf                  # row 2 of sequence 0
    c["kt"][2, :, 4], c["vt"][2, :, 4] = np.nan, np.nan      # sequence 2 sees NaN
    call = Call(c, dev)
    call()
    got, ref = call.out.cpu().numpy().reshape(12, 8, 64), _reference(c)[0]
    bad = [2, 6, 7, 8]
    for r in range(12):
        if r in bad:
            assert np.isnan(got[r]).all() and np.isnan(ref[r]).all()
        else:
            assert_close(got[r], ref[r], f"row {r}", ATTN_TOL)


@pytest.mark.parametrize("plen", [40, 400])
def test_nan_in_a_prompt_that_is_seen(dev, plen):  # noqa: F811
    """NaN for the prompt's sequences and the row's KV head alone."""
    c = _attn_case(18, nh=4, nkv=2, dqk=64, dv=64, plen=[plen, plen], tlen=[3, 0, 9, 5])
    c["kpre"][1, 0, 30, 3] = np.nan
    call = Call(c, dev)
    call()
    got, ref = call.out.cpu().numpy().reshape(4, 4, 64), np.array(_reference(c)[0])
    assert np.isnan(got[2:, :2]).all()
    assert_close(got[:2], ref[:2], "other prompt", ATTN_TOL)
    assert_close(got[2:, 2:], ref[2:, 2:], "other KV head", ATTN_TOL)


@pytest.mark.parametrize("tail", [40, 900])
def test_infinite_logits_and_values_of_a_tail(dev, tail):  # noqa: F811
    """Tails are read as they are: -infinity hides a key, infinity in V stays infinity."""
    c = _attn_case(19, nh=4, nkv=2, dqk=64, dv=64, plen=[90], tlen=[tail, tail], norm=False, rot=0)
    c["qp"] = np.abs(c["qp"])
    c["kt"][0, 0, 7] = -np.inf
    c["vt"][0, 0, 7] = 5
    c["vt"][1, 1, 9, 11] = np.inf
    call = Call(c, dev)
    call()
    got = call.out.cpu().numpy().reshape(2, 4, 64)
    c["kt"][0, 0, 7], c["vt"][1, 1, 9, 11] = -1e4, 0
    ref = np.array(_reference(c)[0])
    assert (got[1, 2:, 11] == np.inf).all()
    got[1, 2:, 11] = ref[1, 2:, 11]
    assert_close(got, ref, "out", ATTN_TOL)


@pytest.mark.parametrize("scale", [1e-15, 1e3])
def test_magnitudes(dev, scale):  # noqa: F811
    c = _attn_case(20, nh=8, nkv=2, dqk=128, dv=128, plen=[300], tlen=[80, 3], norm=False)
    for n in ("vpre", "vt", "vp"):
        c[n] *= np.float32(scale)
    c["kpre"][:, :, 12] = 0
    c["qp"][1] *= np.float32(1e-6)
    call = Call(c, dev)
    call()
    call.check()


def test_large_logits(dev):  # noqa: F811
    """Twelve times the logits that the tolerance is derived for, and so twelve times the tolerance."""
    c = _attn_case(21, nh=8, nkv=2, dqk=128, dv=128, plen=[300], tlen=[500, 3], norm=False)
    c["qp"] *= np.float32(12)
    call = Call(c, dev)
    call()
    call.check(tol=12 * ATTN_TOL)


@pytest.mark.parametrize("plen,tlen,near", [([101], [4], ([100], [4])), ([-3], [4], ([0], [4])), ([90], [11], ([90], [10])),
                                            ([2 ** 31 - 1], [2 ** 31 - 1], ([100], [10]))])
def test_lengths_outside_their_range(dev, plen, tlen, near):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    c = _attn_case(22, nh=4, nkv=2, dqk=64, dv=64, plen=[100], tlen=[10])
    call = Call(c, dev)
    call.plen.copy_(torch.tensor(plen))
    call.tlen.copy_(torch.tensor(tlen))
    call()
    torch.cuda.synchronize()
    assert M.mtp_workspace_status(call.ws) == 7
    c["plen"], c["tlen"] = near
    got = call.out.cpu().numpy().reshape(1, 4, 64)
    assert_close(got, np.array(_reference(c)[0]), "nearest lengths", ATTN_TOL)


def test_captured_calls_on_new_lengths_and_two_streams(dev):  # noqa: F811
    """Graphs of two calls on one workspace, replayed as lengths grow; the same calls on two streams at once."""
    import torch
    import mtp_speculative_draft_gb300 as M
    a = _attn_case(23, nh=8, nkv=2, dqk=128, dv=128, plen=[600], tlen=[5, 20, 60], loose=(0, 10))
    b = _attn_case(24, nh=16, nkv=2, dqk=256, dv=256, plen=[50, 90], tlen=[7, 0], window=40, loose=(0, 10))
    calls = [Call(a, dev), Call(b, dev)]
    own = [c.ws for c in calls]
    for c in calls:
        c()  # whatever a first call sets up
    torch.cuda.synchronize()
    ws = max(own, key=lambda t: t.numel())
    graphs = []
    for c in calls:
        c.ws = ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for grow in (0, 3, 10):
        for c in calls:
            c.c["tlen"] = [t + grow for t in c.c["tlen"]] if grow else c.c["tlen"]
            for n in ("kt", "vt"):  # the rows that the tails have grown by
                x = np.random.default_rng(grow).standard_normal(c.c[n].shape).astype(np.float32)
                at = (np.arange(x.shape[2]) < np.array(c.c["tlen"])[:, None])[:, None, :, None]
                c.c[n] = np.where(at, x, np.float32(np.nan))
                getattr(c, n).copy_(_t(c.c[n], dev))
            c.tlen.copy_(_t(np.array(c.c["tlen"], np.int32), dev))
            c.out.fill_(7.0)
        graphs[0].replay()
        graphs[1].replay()
        for c in calls:
            c.check(f"grown by {grow}")
        if grow == 3:
            break
    side = [torch.cuda.Stream() for _ in calls]
    for c, w in zip(calls, own):
        c.ws = w
        c.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, side):
            c(s)
    torch.cuda.synchronize()
    for c in calls:
        c.check("two streams")
    assert M.mtp_workspace_status(own[0]) == 0


def test_attention_wrapper_refuses(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    call = Call(_attn_case(25, nh=4, nkv=2, dqk=64, dv=64, plen=[10], tlen=[3, 4]), dev)
    good = {k: getattr(call, k) for k in ("qp", "kp", "out", "kt", "vt", "kpre", "vpre", "rope")}
    for name, bad, error in (
            ("qp", call.qp[:1].expand(2, -1), ValueError), ("qp", call.qp.double(), TypeError), ("kp", call.kp[:1], ValueError),
            ("kp", call.kp.cpu(), ValueError), ("out", call.out[:1], ValueError), ("out", call.out.half(), TypeError),
            ("kt", call.kt[:1], ValueError), ("kt", call.kt.transpose(1, 2), ValueError), ("vt", call.vt[..., :32], ValueError),
            ("kt", call.kt[:, :, :4].contiguous(), (ValueError, M._lib.MtpError)), ("kpre", None, ValueError),
            ("kpre", call.kpre[0], ValueError), ("vpre", call.vpre.half(), TypeError),
            ("kpre", call.kpre[:, :, :5].contiguous(), (ValueError, M._lib.MtpError)), ("rope", None, M._lib.MtpError),
            ("rope", call.rope[:64], M._lib.MtpError)):
        for key, value in {**good, name: bad}.items():
            setattr(call, key, value)
        with pytest.raises(error):
            call()
    for key, value in good.items():
        setattr(call, key, value)
    for args in ((call.plen.long(), call.tlen, 1, 1), (call.plen, call.tlen.cpu(), 1, 1), (call.plen, call.tlen, 2 ** 31, 1),
                 (call.plen, call.tlen[::2], 1, 1) if call.tlen[::2].is_contiguous() is False else (call.plen, call.tlen.float(), 1, 1)):
        with pytest.raises((ValueError, TypeError)):
            M.prefix_batch(*args)
    call()
    call.check()


# ------------------------------------------------------------------ beam_select
def _beams(seed, seqs, beams, vocab, done=False, alpha=0.0, spread=1.0):
    rng = np.random.default_rng(seed)
    n = seqs * beams
    x = (3 * rng.standard_normal((n, vocab))).astype(np.float32)
    score = (-20 - spread * rng.random(n)).astype(np.float32)
    length = rng.integers(5, 40, n).astype(np.int32)
    fin = (rng.random(n) < 0.3).astype(np.int32) if done else None
    return dict(x=x, seqs=seqs, beams=beams, score=score, length=length, done=fin, eos=min(2, vocab - 1), alpha=alpha)


class Select:
    """Device copies of a case's inputs and its call; ``shift``: values in front of the first row, ``pad``: behind each."""

    def __init__(self, c, k, dev, shift=0, pad=0):  # noqa: F811
        import torch
        import mtp_speculative_draft_gb300 as M
        self.c, self.k = c, k
        n, V = c["x"].shape
        buf = torch.full((shift + n * (V + pad) + 4,), float("nan"), device=dev)
        self.x = buf[shift:shift + n * (V + pad)].view(n, V + pad)[:, :V]
        self.x.copy_(_t(c["x"], dev))
        self.score, self.length, self.done = _t(c["score"], dev), _t(c["length"], dev), _t(c["done"], dev)
        self.set = M.beam_set(c["seqs"], c["beams"], V, self.score, self.length, self.done, c["eos"], c["alpha"])
        i = lambda: torch.full((c["seqs"], k), -9, dtype=torch.int32, device=dev)  # noqa: E731
        self.parent, self.token, self.new_length, self.new_done = i(), i(), i(), i()
        self.new_score = torch.full((c["seqs"], k), 9.0, device=dev)
        self.ws = M.workspace(M.beam_select_workspace_bytes(self.set, k))

    def __call__(self, stream=None):
        import mtp_speculative_draft_gb300 as M
        M.beam_select(self.set, self.x, self.k, self.parent, self.token, self.new_score, self.new_length, self.new_done, self.ws,
                      stream)

    def check(self, name=""):
        import torch
        import mtp_speculative_draft_gb300 as M
        torch.cuda.synchronize()
        assert M.mtp_workspace_status(self.ws) == 0
        c, B_ = self.c, self.c["beams"]
        got = [t.cpu().numpy() for t in (self.parent, self.token, self.new_score, self.new_length, self.new_done)]
        for s in range(c["seqs"]):
            at = slice(s * B_, s * B_ + B_)
            part = lambda a: None if a is None else a[at]  # noqa: E731
            ref = B.beam_candidates(c["x"][at], c["score"][at], part(c["length"]), part(c["done"]), c["eos"], c["alpha"])
            same_norm = {}  # beams whose ranks are worked out from the same numbers
            for b in range(B_):
                same_norm[b] = (c["x"][s * B_ + b].tobytes(), float(c["score"][s * B_ + b]), int(c["length"][s * B_ + b]))
            near = lambda a, b: (same_norm[a[1]] != same_norm[b[1]] and  # noqa: E731
                                 abs(a[0] - b[0]) <= 2 * SUM_TOL * max(abs(a[0] / a[3]) if a[3] else 1, abs(b[0] / b[3]) if b[3] else 1))
            left = list(ref)
            for j in range(self.k):
                row = [g[s, j] for g in got]
                if not left:
                    assert row[0] == row[1] == -1 and row[2] == -np.inf and row[3] == row[4] == 0, (name, s, j)
                    continue
                i = next((i for i, r in enumerate(left[:40]) if (r[1], r[2]) == (row[0], row[1])), None)
                assert i is not None, (name, s, j, row, left[:3])
                assert all(near(left[i], left[h]) for h in range(i)), (name, s, j, row, left[:i + 1])
                r = left.pop(i)
                assert abs(row[2] - r[3]) <= SUM_TOL + 2.0 ** -24 * abs(r[3]) and (row[3], row[4]) == (r[4], r[5]), (name, s, j, row, r)


@pytest.mark.parametrize("seqs,beams,vocab,k", [
    (1, 1, 1, 1), (1, 1, 1, 3), (1, 1, 7, 5), (1, 4, 4096, 4), (2, 3, 1000, 6), (1, 5, 8189, 10), (1, 2, 8193, 128),
    (3, 4, 16384, 8), (1, 8, 40000, 16), (5, 1, 20001, 1), (1, 64, 300, 128), (16, 64, 50, 64), (4, 7, 999, 100), (1, 3, 2, 9)])
@pytest.mark.parametrize("alpha,done", [(0.0, False), (0.7, True)])
def test_selection(dev, seqs, beams, vocab, k, alpha, done):  # noqa: F811
    call = Select(_beams(vocab + k, seqs, beams, vocab, done, alpha), k, dev, shift=vocab % 4, pad=beams % 4)
    call()
    call.check()


def test_selection_of_a_large_vocabulary(dev):  # noqa: F811
    """Rows at every alignment; the best tokens at both ends of the row and of its chunks."""
    c = _beams(5, 1, 4, 152577)
    for r, toks in enumerate(([0, 152576], [8191, 8192], [1, 2, 3], [152573, 152575])):
        c["x"][r, toks] = 40 + np.arange(len(toks), dtype=np.float32)
    for shift in range(4):
        call = Select(c, 12, dev, shift=shift)
        call()
        call.check(f"shift {shift}")


@pytest.mark.parametrize("vocab,k", [(300, 5), (9000, 128), (50000, 16)])
def test_equal_logits(dev, vocab, k):  # noqa: F811
    """Constant rows, rows of few values, -0 beside 0: the lowest tokens, and the lower beam among equal ones."""
    c = _beams(6, 1, 6, vocab)
    c["x"][0], c["x"][1] = 2.5, -0.0
    c["x"][1, ::3] = 0.0
    c["x"][2:4] = np.random.default_rng(1).integers(0, 3, vocab)  # two beams alike
    c["x"][4, 7:] = -np.inf
    c["score"][2:4], c["length"][2:4] = -20, 9
    call = Select(c, k, dev)
    call()
    call.check()


def test_equal_ranks_of_many_beams(dev):  # noqa: F811
    """64 beams alike and constant: 8192 equal candidates, and 300 tokens of one beam behind 40 better ones."""
    c = _beams(7, 2, 64, 1000)
    c["x"][:64], c["score"][:64], c["length"][:64] = 1.0, -3.0, 4
    c["x"][64:] = -1.0
    c["x"][64:104, 500] = np.arange(40, dtype=np.float32)
    c["score"][64:], c["length"][64:] = -3.0, 4
    call = Select(c, 128, dev)
    call()
    call.check()
    assert call.parent[0].tolist() == [0] * 128 and call.token[0].tolist() == list(range(128))


def test_beams_that_offer_nothing(dev):  # noqa: F811
    """Scores that are not finite, masked rows, infinity and NaN in a row, fewer candidates than wanted."""
    c = _beams(8, 2, 6, 90)
    c["score"][[0, 1, 2]] = -np.inf, np.nan, np.inf
    c["x"][3] = -np.inf
    c["x"][4, 5] = np.inf
    c["x"][5], c["x"][5, [8, 60]] = np.nan, 1.0
    c["score"][6:] = -np.inf
    call = Select(c, 7, dev)
    call()
    call.check()
    assert call.token[0].tolist() == [8, 60, -1, -1, -1, -1, -1] and (call.parent[1] == -1).all()


def test_the_first_step_of_a_search(dev):  # noqa: F811
    """One beam at 0, the others at -infinity."""
    c = _beams(9, 3, 4, 5000)
    c["score"] = np.where(np.arange(12) % 4 == 0, 0, -np.inf).astype(np.float32)
    c["length"][:] = 0
    call = Select(c, 4, dev)
    call()
    call.check()
    assert (call.parent == 0).all() and (call.new_length == 1).all()


@pytest.mark.parametrize("alpha", [-1.0, 1.0, 300.0, -300.0])
def test_finished_beams_and_lengths(dev, alpha):  # noqa: F811
    """Finished beams of length 0, negative lengths, penalties of any size; every beam finished."""
    c = _beams(10, 2, 4, 600, alpha=alpha)
    c["done"] = np.array([0, 1, 0, 1, 1, 1, 1, 1], np.int32) * 3
    c["length"] = np.array([1, 0, -5, 9, 1, 2, 3, 4], np.int32)
    if abs(alpha) > 1:
        c["length"][:4] = 1, 0, 0, 1  # 2^300 and less; ranks of 1e+-90 and more
    call = Select(c, 4, dev)
    call()
    call.check()


def test_extreme_logits(dev):  # noqa: F811
    """Logits of any size: exponentials that underflow, a row of one token, differences below a step."""
    c = _beams(11, 1, 6, 9000)
    c["x"][0] *= np.float32(1e4)
    c["x"][1] -= np.float32(1e30)
    c["x"][2] = np.float32(3e38)
    c["x"][3] = np.where(np.arange(9000) == 4000, 0, -np.inf)
    c["x"][4] *= np.float32(1e-30)
    call = Select(c, 20, dev)
    call()
    call.check()


def test_selection_in_place_captured_and_without_lengths(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    c = _beams(12, 4, 5, 12000, done=True, alpha=0.5)
    a, b = Select(c, 5, dev), Select(c, 5, dev)
    a()
    M.beam_select(b.set, b.x, 5, b.parent, b.token, b.score, b.length, b.done, b.ws)
    for x, y in ((a.parent, b.parent), (a.token, b.token), (a.new_score, b.score), (a.new_length, b.length), (a.new_done, b.done)):
        assert torch.equal(x.view(-1), y.view(-1))
    plain = M.beam_set(4, 5, 12000, a.score)
    M.beam_select(plain, a.x, 5, a.parent, a.token, a.new_score, ws=a.ws)
    ref = B.beam_select(c["x"], 4, 5, 5, c["score"])
    assert a.token.tolist() == ref[1].tolist()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    d = Select(_beams(13, 3, 4, 9001), 6, dev)
    d()
    with torch.cuda.graph(g):
        d()
    for seed in (14, 15):
        d.c = _beams(seed, 3, 4, 9001)
        d.x.copy_(_t(d.c["x"], dev))
        d.score.copy_(_t(d.c["score"], dev))
        d.length.copy_(_t(d.c["length"], dev))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
            g.replay()
        side.synchronize()
        d.check(f"replayed on seed {seed}")


def test_selection_wrapper_refuses(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    s = Select(_beams(16, 2, 3, 100), 3, dev)
    args = [s.x, 3, s.parent, s.token, s.new_score, s.new_length, s.new_done]
    for i, bad, error in ((0, s.x[:5], ValueError), (0, s.x[:, :99], ValueError), (0, s.x.half(), TypeError), (0, s.x.cpu(), ValueError),
                          (1, 0, M._lib.MtpError), (1, 2 ** 40, ValueError), (2, s.parent.long(), TypeError), (3, s.token[:1], ValueError),
                          (4, s.new_score.double(), TypeError), (5, s.length, M._lib.MtpError), (6, s.new_length, M._lib.MtpError)):
        a = list(args)
        a[i] = bad
        if i == 5:
            a[1] = 2  # in place needs as many candidates as beams
        with pytest.raises(error):
            M.beam_select(s.set, *a, ws=s.ws)
    with pytest.raises(ValueError):
        M.beam_set(2, 4, 100, s.score)
    with pytest.raises(TypeError):
        M.beam_set(2, 3, 100, s.score, s.length.long())
    s()
    s.check()


# ------------------------------------------------------------------ kv_beam_reorder
@pytest.mark.parametrize("seqs,beams,layers,nkv,dqk,dv,tail", [
    (1, 1, 1, 1, 4, 4, 1), (1, 2, 1, 1, 32, 64, 7), (3, 4, 2, 2, 64, 32, 33), (1, 64, 1, 2, 256, 256, 5), (2, 5, 70, 1, 20, 8, 9),
    (1, 3, 2, 3, 128, 128, 700), (100, 10, 1, 1, 8, 12, 3)])
@pytest.mark.parametrize("kind", ["random", "swap", "first", "stay"])
def test_reorder(dev, seqs, beams, layers, nkv, dqk, dv, tail, kind):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    rng = np.random.default_rng(seqs + beams + tail)
    n, cap = seqs * beams, tail + 3
    parent = {"random": rng.integers(-1, beams, (seqs, beams)), "swap": np.tile(np.arange(beams)[::-1], (seqs, 1)),
              "first": np.zeros((seqs, beams)), "stay": np.tile(np.arange(beams), (seqs, 1))}[kind].astype(np.int32)
    length = rng.integers(-1, tail + 1, n).astype(np.int32)
    length[0] = tail
    k = [rng.standard_normal((n, nkv, cap, dqk)).astype(np.float32) for _ in range(layers)]
    v = [rng.standard_normal((n, nkv, cap, dv)).astype(np.float32) for _ in range(layers)]
    tk, tv = [_t(x, dev) for x in k], [_t(x, dev) for x in v]
    ws = M.kv_beam_reorder(M.kv_tails(tk, tv, beams), _t(parent, dev), _t(length, dev), tail)
    torch.cuda.synchronize()
    assert M.mtp_workspace_status(ws) == 0
    for x, y in zip(k + v, tk + tv):
        np.testing.assert_array_equal(y.cpu().numpy(), B.beam_reorder(x, parent, length, beams))


def test_reorder_parents_and_lengths_outside_their_range(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    k = np.random.default_rng(3).standard_normal((4, 2, 9, 16)).astype(np.float32)
    for parent, length, near in (([1, 0, 4, -7], [3, 3, 3, 3], ([1, 0, -1, -1], [3, 3, 3, 3])),
                                 ([1, 0, 3, 2], [3, 9, 2 ** 31 - 1, -2 ** 31], ([1, 0, 3, 2], [3, 8, 8, 0]))):
        tk, ws = _t(k, dev), M.workspace(M.kv_beam_workspace_bytes())
        tv = tk.clone()
        M.kv_beam_reorder(M.kv_tails([tk], [tv], 4), _t(np.array(parent, np.int32), dev), _t(np.array(length, np.int32), dev), 8, ws)
        torch.cuda.synchronize()
        assert M.mtp_workspace_status(ws) == 7
        np.testing.assert_array_equal(tk.cpu().numpy(), B.beam_reorder(k, [near[0]], near[1], 4))
        assert torch.equal(tk, tv)


def test_reorder_offsets_past_32_bits(dev):  # noqa: F811
    """The second beam's rows start 2^31 values behind the first's."""
    import torch
    import mtp_speculative_draft_gb300 as M
    cap = 1 << 26
    k, v = torch.empty(2, 1, cap, 32, device=dev), torch.empty(2, 1, 8, 32, device=dev)
    v = torch.empty(2, 1, cap, 32, device=dev)
    for x in (k, v):
        x[:, :, :8] = torch.randn(2, 1, 8, 32, device=dev)
        x[:, :, cap - 4:] = torch.randn(2, 1, 4, 32, device=dev)
    want = [(x[1, :, :5].clone(), x[0, :, 5:8].clone(), x[0, :, :5].clone(), x[1, :, 5:8].clone()) for x in (k, v)]
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    M.kv_beam_reorder(M.kv_tails([k], [v], 2), i(1, 0), i(5, 5), 8)
    for x, (a, b, c, d) in zip((k, v), want):
        assert torch.equal(x[0, :, :5], a) and torch.equal(x[0, :, 5:8], b) and torch.equal(x[1, :, :5], c) and torch.equal(x[1, :, 5:8], d)


def test_reorder_wrapper_refuses(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    k, v = torch.randn(6, 2, 9, 16, device=dev), torch.randn(6, 2, 9, 16, device=dev)
    for args in (([k], [v, v], 3), ([k], [k], 3), ([k, k], [v, v], 3), ([k], [v], 4), ([k], [v], 0), ([k[0]], [v[0]], 2),
                 ([k], [v[:, :1]], 3), ([k.transpose(1, 2)], [v], 3), ([], [], 1)):
        with pytest.raises((ValueError, TypeError)):
            M.kv_tails(*args)
    t = M.kv_tails([k], [v], 3)
    i = torch.zeros(6, dtype=torch.int32, device=dev)
    for args, error in (((i[:5], i, 3), ValueError), ((i.long(), i, 3), TypeError), ((i, i, 10), M._lib.MtpError),
                        ((i, i, 2 ** 33), ValueError), ((i, i.cpu(), 3), ValueError)):
        with pytest.raises(error):
            M.kv_beam_reorder(t, *args)


# ------------------------------------------------------------------ a search
@pytest.mark.parametrize("captured", [False, True])
def test_a_beam_search(dev, captured):  # noqa: F811
    """Two prompts of four beams through two attention layers, seven steps, the step's calls captured once or not,
    against a search that computes every hypothesis from its tokens alone in 64 bits."""
    import torch
    import mtp_speculative_draft_gb300 as M
    rng = np.random.default_rng(31)
    nh, nkv, d, V, layers, steps, beams, plen, alpha, eos = 4, 2, 32, 301, 2, 7, 4, [90, 70], 0.6, 5
    n, tmax, theta = len(plen) * beams, steps, 1e4
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    embed = f(V, nh * d)
    W = [dict(q=f(nh * d, nh * d) / 12, k=f(nh * d, nkv * d) / 12, v=f(nh * d, nkv * d) / 6) for _ in range(layers)]
    head, sink = f(nh * d, V) / 3, f(nh)
    head[:, eos] += np.float32(0.08)
    pre = [(f(2, nkv, max(plen), d), f(2, nkv, max(plen), d)) for _ in range(layers)]
    start = np.array([[7] * beams, [11] * beams], np.int32).ravel()

    # --- the calls
    up = lambda a: _t(a, dev)  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    g = M.attn_geom(nh, nkv, d, d)
    tok, parent, done = up(start), i32([0] * n), i32([0] * n)
    score = up(np.where(np.arange(n) % beams == 0, 0, -np.inf).astype(np.float32))
    tlen = i32([0] * n)
    tails = [(torch.full((n, nkv, tmax + 1, d), float("nan"), device=dev), torch.full((n, nkv, tmax + 1, d), float("nan"), device=dev))
             for _ in range(layers)]
    batch = M.prefix_batch(i32(plen), tlen, max(plen), tmax)
    sel = M.beam_set(len(plen), beams, V, score, tlen, done, eos, alpha)  # a tail's rows are the beam's tokens
    moves = M.kv_tails([k for k, _ in tails], [v for _, v in tails], beams)
    rope, out = _table(max(plen) + tmax + 1, d, theta, dev), torch.zeros(n, nh * d, device=dev)
    ws = M.workspace(max(M.attn_prefix_sink_workspace_bytes(g, batch), M.beam_select_workspace_bytes(sel, beams)))
    dW = [{k: up(w) for k, w in x.items()} for x in W]
    dpre, dembed, dhead, dsink = [(up(k), up(v)) for k, v in pre], up(embed), up(head), up(sink)
    logits = torch.empty(n, V, device=dev)

    def step():
        x = dembed[tok.long()]
        for w, (kp, vp), (kt, vt) in zip(dW, dpre, tails):
            M.attn_prefix_sink(g, batch, x @ w["q"], x @ w["k"], x @ w["v"], None, None, rope, dsink, kp, vp, kt, vt, out, ws)
            x = x + out
        torch.matmul(x, dhead, out=logits)
        M.beam_select(sel, logits, beams, parent, tok, score, tlen, done, ws)
        M.kv_beam_reorder(moves, parent, tlen, tmax, ws)

    allow = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    history, graph = [], None
    try:
        for s in range(steps):
            if captured and s == 1:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            if graph is not None:
                graph.replay()
            else:
                step()
            torch.cuda.synchronize()
            history.append([t.cpu().numpy().copy() for t in (parent, tok, score, tlen, done)])
    finally:
        torch.backends.cuda.matmul.allow_tf32 = allow
    assert M.mtp_workspace_status(ws) == 0

    # --- the same search from whole hypotheses, in 64 bits
    def forward(p, tokens):
        """Logits of the last token: a hypothesis' tokens one after another over the prompt's rows."""
        K, Vv = ([x[p, :, :plen[p]].astype(np.float64) for x in side] for side in zip(*pre))
        for j, t in enumerate(tokens):
            x = embed[t].astype(np.float64)
            for l, w in enumerate(W):
                pos = [[plen[p] + j]]
                q = T.rope_axes((x @ w["q"].astype(np.float64)).reshape(1, nh, d), pos, (d // 2,), False, theta)[0]
                k = T.rope_axes((x @ w["k"].astype(np.float64)).reshape(1, nkv, d), pos, (d // 2,), False, theta)[0]
                K[l] = np.concatenate([K[l], k[:, None]], 1)
                Vv[l] = np.concatenate([Vv[l], (x @ w["v"].astype(np.float64)).reshape(nkv, 1, d)], 1)
                o = np.zeros((nh, d))
                for h in range(nh):
                    lg = K[l][h // 2] @ q[h] / math.sqrt(d)
                    e = np.exp(lg - max(lg.max(), sink[h]))
                    o[h] = e @ Vv[l][h // 2] / (e.sum() + math.exp(sink[h] - max(lg.max(), sink[h])))
                x = x + o.ravel()
        return x @ head.astype(np.float64)

    for p in range(2):
        hyps = [([int(start[p * beams])], 0.0 if b == 0 else -np.inf, 0, 0) for b in range(beams)]
        for s in range(steps):
            x = np.array([forward(p, h[0]) if np.isfinite(h[1]) and not h[3] else np.zeros(V) for h in hyps])
            cands = B.beam_candidates(x, [h[1] for h in hyps], [h[2] for h in hyps], [h[3] for h in hyps], eos, alpha)
            # float32 products and attention of two layers: logits of order 10 are off by 1e-4 at most, ranks by less
            assert all(a[0] - b[0] > 1e-4 for a, b in zip(cands[:beams], cands[1:beams + 1])), "the test's own near tie"
            at = slice(p * beams, p * beams + beams)
            gp, gt, gs, gl, gd = (a[at] for a in history[s])
            assert gp.tolist() == [c[1] for c in cands[:beams]] and gt.tolist() == [c[2] for c in cands[:beams]], (p, s)
            assert gl.tolist() == [c[4] for c in cands[:beams]] and gd.tolist() == [c[5] for c in cands[:beams]]
            np.testing.assert_allclose(gs, [c[3] for c in cands[:beams]], atol=2e-4 * (s + 1))
            hyps = [(hyps[c[1]][0] + ([] if hyps[c[1]][3] else [c[2]]), c[3], c[4], c[5]) for c in cands[:beams]]
    assert any(h[4].any() for h in history)  # some hypothesis has ended
