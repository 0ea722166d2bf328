"""Attention over shared prompts where the launches are three (prep, split, tail), and where a size decides that they
are one.  Tolerances as in test_gpu_beams.py."""

import numpy as np
import pytest

from helpers import assert_close
from oracle import beam_oracle as B
from oracle import tree_oracle as T
from test_gpu_beams import ATTN_TOL, Call, _attn_case, _reference, dev  # noqa: F401
from test_gpu_tree import _t

pytestmark = pytest.mark.gpu


def test_most_prompts_of_most_kv_heads(dev):  # noqa: F811
    """1024 prompts of 64 KV heads, one more than a grid's third axis holds: a few of them against the reference,
    every tail's rows outside the new ones as they were."""
    rng = np.random.default_rng(5)
    c = _attn_case(60, nh=192, nkv=64, dqk=32, dv=32, plen=[int(n) for n in rng.integers(0, 9, 1023)] + [8],
                   tlen=[int(t) for t in rng.integers(-1, 4, 1023)] + [3], m=2)
    call = Call(c, dev)
    call()
    got, m = call.out.cpu().numpy().reshape(1024, 2, 192, 32), 2
    kt, vt = call.kt.cpu().numpy(), call.vt.cpu().numpy()
    pick = [0, 1, 511, 512, 1022, 1023]
    rows = np.concatenate([np.arange(b * m, b * m + m) for b in pick])
    sub = {**c, **{n: [c[n][b] for b in pick] for n in ("plen", "tlen")}, **{n: c[n][pick] for n in ("kpre", "vpre", "kt", "vt")},
           **{n: c[n][rows] for n in ("qp", "kp", "vp")}}
    ref, k, _ = _reference(sub)
    for x, b in enumerate(pick):
        t = c["tlen"][b]
        if t >= 0:
            assert_close(got[b], np.array(ref[x * m:x * m + m]), f"sequence {b}", ATTN_TOL)
            assert_close(kt[b, :, t:t + m], k[x * m:x * m + m].transpose(1, 0, 2), f"keys of {b}", 2e-6)
    for b, t in enumerate(c["tlen"]):
        keep = np.ones(kt.shape[2], bool)
        if t >= 0:
            keep[t:t + m] = False
            np.testing.assert_array_equal(vt[b, :, t:t + m], c["vp"][b * m:b * m + m].reshape(m, 64, 32).transpose(1, 0, 2))
        else:
            assert (got[b] == 7).all()
        np.testing.assert_array_equal(kt[b][:, keep], c["kt"][b][:, keep])
        np.testing.assert_array_equal(vt[b][:, keep], c["vt"][b][:, keep])


def _launches(call):
    """Kernels that a call launches."""
    import torch
    from mtp_speculative_draft_gb300.api import launch_timing
    events = [torch.cuda.Event(enable_timing=True) for _ in range(8)]
    for e in events:
        e.record()  # makes the event
    with launch_timing(events) as timing:
        call()
    return timing.n - 1


@pytest.mark.parametrize("scale", [1e-15, 1e3])
def test_magnitudes_in_a_long_prompt(dev, scale):  # noqa: F811
    c = _attn_case(61, nh=8, nkv=2, dqk=128, dv=128, plen=[12300], tlen=[80, 3], norm=False)
    for n in ("vpre", "vt", "vp"):
        c[n] *= np.float32(scale)
    c["kpre"][:, :, 12] = 0
    c["kpre"][:, :, 700:900] *= np.float32(1e-3)
    c["qp"][1] *= np.float32(1e-6)
    call = Call(c, dev)
    assert _launches(call) == 3
    call.check()


@pytest.mark.parametrize("dim", [128, 256])
def test_large_logits_over_a_long_prompt(dev, dim):  # noqa: F811
    """Twelve times the logits that the tolerance is derived for, and so twelve times the tolerance."""
    c = _attn_case(62, nh=8, nkv=2, dqk=dim, dv=dim, plen=[12300], tlen=[500, 3], norm=False)
    c["qp"] *= np.float32(12)
    call = Call(c, dev)
    assert _launches(call) == 3
    call.check(tol=12 * ATTN_TOL)


def test_long_prompts_repeat_bit_for_bit(dev):  # noqa: F811
    call = Call(_attn_case(63, nh=40, nkv=8, dqk=128, dv=128, plen=[12300], tlen=[40, 700, 3]), dev)
    assert _launches(call) == 3
    first = call.out.clone()
    for _ in range(3):
        call.out.fill_(3.0)
        call()
        assert (call.out == first).all()


def test_workspace_of_long_prompts_used_by_other_calls_before(dev):  # noqa: F811
    """Three-launch calls of two geometries, rules and selections on one workspace that held NaN."""
    import torch
    import mtp_speculative_draft_gb300 as M
    a = Call(_attn_case(64, nh=16, nkv=1, dqk=256, dv=256, plen=[12400], tlen=[9, 30, 2]), dev)
    b = Call(_attn_case(65, nh=5, nkv=1, dqk=96, dv=96, plen=[12300, 40], tlen=[2, 900]), dev)
    x = np.random.default_rng(4).standard_normal((64, 9001)).astype(np.float32)
    logits, want = _t(x, dev), [t for t, _ in T.greedy(x)]
    tok, val = torch.empty(64, dtype=torch.int32, device=dev), torch.empty(64, device=dev)
    out = [torch.empty(8, 8, dtype=d, device=dev) for d in (torch.int32, torch.int32, torch.float32)]
    beams = M.beam_set(8, 8, 9001, torch.zeros(64, device=dev))
    ref = B.beam_select(x, 8, 8, 8, np.zeros(64))
    ws = M.workspace(max(a.ws.numel(), b.ws.numel(), M.logit_rules_argmax_workspace_bytes(64),
                         M.beam_select_workspace_bytes(beams, 8)))
    a.ws = b.ws = ws
    ws[1024 + 16384:] = 255  # NaN behind the header and the rules' joins
    assert _launches(a) == _launches(b) == 3
    for _ in range(2):
        for call in (a, b):
            call.kt.copy_(_t(call.c["kt"], dev))
            call.vt.copy_(_t(call.c["vt"], dev))
            call.out.fill_(7.0)
            call()
            call.check()
            M.logit_rules_argmax(M.logit_rules(9001), logits, tok, val, None, ws)
            assert tok.tolist() == want
            M.beam_select(beams, logits, 8, *out, ws=ws)
            assert out[1].tolist() == ref[1].tolist()


def _grow(c, grow):
    """The case with tails longer by `grow` rows, and its rows."""
    rng = np.random.default_rng(grow)
    c["tlen"] = [t + grow for t in c["tlen"]]
    for n in ("kt", "vt"):
        at = (np.arange(c[n].shape[2]) < np.array(c["tlen"])[:, None])[:, None, :, None]
        c[n] = np.where(at, rng.standard_normal(c[n].shape).astype(np.float32), np.float32(np.nan))


def test_captured_long_prompts_on_new_lengths_and_two_streams(dev):  # noqa: F811
    """Graphs of two three-launch calls on one workspace, replayed as tails grow and as prompts get other lengths; the
    same calls on two streams at once."""
    import torch
    import mtp_speculative_draft_gb300 as M
    calls = [Call(_attn_case(66, nh=8, nkv=2, dqk=128, dv=128, plen=[12350], tlen=[5, 20, 60], loose=(0, 10)), dev),
             Call(_attn_case(67, nh=16, nkv=2, dqk=256, dv=256, plen=[12300, 90], tlen=[7, 0], window=12290, m=2,
                             loose=(0, 10)), dev)]
    own = [c.ws for c in calls]
    for c in calls:
        assert _launches(c) == 3
    torch.cuda.synchronize()
    ws = max(own, key=lambda t: t.numel())
    graphs = []
    for c in calls:
        c.ws = ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for grow, cut in ((0, 0), (3, 0), (7, 700)):
        for c in calls:
            _grow(c.c, grow)
            c.c["plen"] = [max(0, p - cut) for p in c.c["plen"]]
            for n in ("kt", "vt"):
                getattr(c, n).copy_(_t(c.c[n], dev))
            c.tlen.copy_(_t(np.array(c.c["tlen"], np.int32), dev))
            c.plen.copy_(_t(np.array(c.c["plen"], np.int32), dev))
            c.out.fill_(7.0)
        graphs[0].replay()
        graphs[1].replay()
        for c in calls:
            c.check(f"grown by {grow}")
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
    assert M.mtp_workspace_status(own[0]) == M.mtp_workspace_status(own[1]) == 0
