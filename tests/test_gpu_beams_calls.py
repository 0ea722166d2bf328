"""The beam search's step as a program may call it: long prompts (three launches) beside short ones (one), first calls
under capture, two calls at once, workspaces passed around, lengths at the ends of their ranges."""

import numpy as np
import pytest

from helpers import assert_close
from oracle import beam_oracle as B
from oracle import tree_oracle as T
from test_gpu_beams import ATTN_TOL, Call, Select, _attn_case, _beams, _reference, dev  # noqa: F401
from test_gpu_tree import _t

pytestmark = pytest.mark.gpu

# more keys than one launch takes
LONG = [
    dict(nh=1, nkv=1, dqk=32, dv=32, plen=[12300], tlen=[0]),
    dict(nh=4, nkv=2, dqk=64, dv=64, plen=[12400, 0, 77], tlen=[5, -1, 9, 0, 64, 7]),          # an empty prompt among others
    dict(nh=2, nkv=2, dqk=64, dv=64, plen=[12300], tlen=[-1, -1, -1]),                         # no sequence at all
    dict(nh=8, nkv=1, dqk=128, dv=128, plen=[12289], tlen=[17, 0, -1, 300], gated=True),
    dict(nh=5, nkv=1, dqk=128, dv=128, plen=[12500], tlen=[9] * 30, gated=True),               # 150 rows: two tiles
    dict(nh=16, nkv=2, dqk=256, dv=256, plen=[12300, 300], tlen=[40, 0, 31, 129], axes=(44, 42, 42)),
    dict(nh=8, nkv=2, dqk=192, dv=128, plen=[13000], tlen=[77, 3, 200], m=4, window=12600, norm=False, sinks=True),
    dict(nh=6, nkv=6, dqk=64, dv=96, plen=[12500], tlen=[3, 0], m=16, window=12450),
    dict(nh=12, nkv=1, dqk=160, dv=224, plen=[12515], tlen=[11, 12, 700], rot=40),
    dict(nh=64, nkv=1, dqk=32, dv=256, plen=[12329], tlen=[3, 90, 1], rot=0),
    dict(nh=128, nkv=2, dqk=32, dv=64, plen=[12400], tlen=[300, 2], m=3),
    dict(nh=3, nkv=3, dqk=32, dv=32, plen=[12331], tlen=[31] * 20, rot=10, sinks=True),
    dict(nh=2, nkv=1, dqk=256, dv=128, plen=[12370], tlen=[1500, 3], loose=(0, 400)),
    dict(nh=4, nkv=1, dqk=64, dv=64, plen=[5, 12400, 6000, 64], tlen=[7, 2, 0, 4], loose=(9000, 0)),
]


@pytest.mark.parametrize("i", range(len(LONG)))
def test_attention_over_long_prompts(dev, i):  # noqa: F811
    call = Call(_attn_case(700 + i, **LONG[i]), dev, pad=4 * (i % 3))
    call()
    call.check(str(LONG[i]))
    first = call.out.clone()
    call.out.fill_(7.0)
    call()
    assert (call.out == first).all()


def test_one_launch_and_three_agree(dev):  # noqa: F811
    """The same batch with a bound that one launch takes, and with one that it does not."""
    outs = []
    for loose in (0, 12288):
        c = _attn_case(5, nh=40, nkv=8, dqk=128, dv=128, plen=[700], tlen=[30, 100, 0], m=2, gated=True, sinks=True)
        c["pmax"] += loose
        for n in ("kpre", "vpre"):
            c[n] = np.pad(c[n], ((0, 0), (0, 0), (0, loose), (0, 0)), constant_values=np.nan)
        call = Call(c, dev)
        call()
        call.check(f"loose by {loose}")
        outs.append((call.out.cpu().numpy(), call.kt.cpu().numpy()))
    assert_close(outs[0][0], outs[1][0], "outputs", 2 * ATTN_TOL)
    np.testing.assert_array_equal(outs[0][1], outs[1][1])


def test_hidden_rows_behind_long_prompts(dev):  # noqa: F811
    """NaN and infinity below a window's edge, in later new rows, in other prompts and sequences."""
    c = _attn_case(6, nh=4, nkv=2, dqk=64, dv=64, plen=[13000, 12900], tlen=[40, 0, 10, 60], m=3, window=12700)
    lo = 13000 + 0 + 1 - 12700                               # the first prompt's row that sequence 1's row 0 still sees
    c["kpre"][0, :, :lo], c["vpre"][0, :, :lo] = np.nan, np.inf
    c["kp"][2], c["vp"][2] = np.nan, np.inf                   # row 2 of sequence 0
    c["vpre"][0, 1, lo + 3] = np.nan                          # an edge that sequence 1 sees and sequence 0 does not
    c["kt"][2, :, 4] = np.nan                                 # sequence 2 sees NaN
    call = Call(c, dev)
    call()
    got, ref = call.out.cpu().numpy().reshape(12, 4, 64), _reference(c)[0]
    for r in range(12):
        nan = np.isnan(ref[r])
        assert (np.isnan(got[r]) == nan).all(), r
        if not nan.all():
            assert_close(got[r][~nan], ref[r][~nan], f"row {r}", ATTN_TOL)
    assert [bool(np.isnan(ref[r]).any()) for r in range(12)] == [False, False, True, True, True, True, True, True, True, False, False, False]


def test_nan_in_a_long_prompt_that_is_seen(dev):  # noqa: F811
    c = _attn_case(7, nh=4, nkv=2, dqk=64, dv=64, plen=[12400, 12400], tlen=[3, 0, 9, 5])
    c["kpre"][1, 0, 30, 3] = np.nan
    call = Call(c, dev)
    call()
    got, ref = call.out.cpu().numpy().reshape(4, 4, 64), np.array(_reference(c)[0])
    assert np.isnan(got[2:, :2]).all()
    assert_close(got[:2], ref[:2], "other prompt", ATTN_TOL)
    assert_close(got[2:, 2:], ref[2:, 2:], "other KV head", ATTN_TOL)


def test_long_prompts_offsets_past_32_bits(dev):  # noqa: F811
    """The second KV head's rows start 2^31 values behind the first's, in a prompt of three launches."""
    import torch
    call = Call(_attn_case(12, nh=4, nkv=2, dqk=32, dv=32, plen=[12400], tlen=[90]), dev)
    cap = 1 << 26
    for name in ("kpre", "vpre"):
        big, small = torch.empty(1, 2, cap, 32, device=dev), getattr(call, name)
        big[:, :, :small.shape[2]] = small
        setattr(call, name, big)
    call()
    call.check()


def test_lengths_outside_their_range_behind_long_prompts(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    c = _attn_case(22, nh=4, nkv=2, dqk=64, dv=64, plen=[12300], tlen=[10, 5])
    call = Call(c, dev)
    call.plen.fill_(12301)
    call.tlen.copy_(torch.tensor([2 ** 31 - 1, 5], dtype=torch.int32))
    call()
    torch.cuda.synchronize()
    assert M.mtp_workspace_status(call.ws) == 7
    assert_close(call.out.cpu().numpy().reshape(2, 4, 64), np.array(_reference(c)[0]), "nearest lengths", ATTN_TOL)


def test_counters_and_joins_of_a_shared_workspace(dev):  # noqa: F811
    """Calls whose parts are counted, between rules of 1024 rows, whose joins lie beside the counters; captured and
    replayed in turn as well."""
    import torch
    import mtp_speculative_draft_gb300 as M
    calls = [Call(_attn_case(31, nh=8, nkv=8, dqk=64, dv=64, plen=[0], tlen=[3000, 2, -1, 1700], sinks=True), dev),
             Call(_attn_case(32, nh=16, nkv=2, dqk=256, dv=256, plen=[900], tlen=[9, 700, 2]), dev),
             Call(_attn_case(33, nh=8, nkv=2, dqk=64, dv=64, plen=[12400], tlen=[900, 3]), dev)]
    x = np.random.default_rng(4).standard_normal((1024, 5001)).astype(np.float32)
    logits, want = _t(x, dev), [t for t, _ in T.greedy(x)]
    tok, val = torch.empty(1024, dtype=torch.int32, device=dev), torch.empty(1024, device=dev)
    ws = M.workspace(max([c.ws.numel() for c in calls] + [M.logit_rules_argmax_workspace_bytes(1024)]))
    rules = M.logit_rules(5001)

    def all_of_them():
        for c in calls:
            c.ws = ws
            c()
            M.logit_rules_argmax(rules, logits, tok, val, None, ws)

    all_of_them()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        all_of_them()
    for _ in range(3):
        tok.fill_(-9)
        for c in calls:
            c.out.fill_(7.0)
        g.replay()
        all_of_them()
        for i, c in enumerate(calls):
            c.check(f"call {i}")
        assert tok.tolist() == want


def test_first_call_of_a_process_is_captured(dev):  # noqa: F811
    """Each call's first launch in a process may be under capture."""
    import os
    import subprocess
    import sys
    code = """
import numpy as np, torch
import test_gpu_beams as G
import mtp_speculative_draft_gb300 as M
from oracle import beam_oracle as B
dev = torch.device("cuda:0")
torch.zeros(1, device=dev)
for kw in (dict(nh=8, nkv=2, dqk=64, dv=64, plen=[12300]), dict(nh=4, nkv=2, dqk=160, dv=128, plen=[300]),
           dict(nh=5, nkv=1, dqk=64, dv=160, plen=[12300])):
    call = G.Call(G._attn_case(3, tlen=[5, 90], norm=False, rot=0, **kw), dev)
    sel = G.Select(G._beams(4, 2, 3, 9000), 3, dev)
    k = np.random.default_rng(1).standard_normal((6, 2, 9, 32)).astype(np.float32)
    tk, tv = G._t(k, dev), G._t(k, dev)
    moves, parent = M.kv_tails([tk], [tv], 3), torch.tensor([1, 2, 0, 0, 0, 1], dtype=torch.int32, device=dev)
    length, ws = torch.full((6,), 8, dtype=torch.int32, device=dev), M.workspace(M.kv_beam_workspace_bytes())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        sel()
        M.kv_beam_reorder(moves, parent, length, 9, ws)
    g.replay()
    call.check()
    sel.check()
    assert (tk.cpu().numpy() == B.beam_reorder(k, [[1, 2, 0], [0, 0, 1]], [8] * 6, 3)).all() and torch.equal(tk, tv)
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([here, os.path.dirname(here)])}
    done = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_calls_on_two_streams_at_once(dev):  # noqa: F811
    """Selections and moves of their own workspaces, interleaved on two streams."""
    import torch
    import mtp_speculative_draft_gb300 as M
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    sel = [Select(_beams(60 + i, 4 - i, 5, 30000 + i, done=True, alpha=0.7), 7, dev, shift=i) for i in range(2)]
    rng = np.random.default_rng(3)
    k = [rng.standard_normal((4, 2, 50, 64)).astype(np.float32) for _ in side]
    t = [_t(x, dev) for x in k]
    tails = [M.kv_tails([x], [x.clone()], 2) for x in t]
    swap, length = torch.tensor([1, 0, 1, 0], dtype=torch.int32, device=dev), torch.full((4,), 41, dtype=torch.int32, device=dev)
    ws = [M.workspace(M.kv_beam_workspace_bytes()) for _ in side]
    torch.cuda.synchronize()
    for _ in range(25):  # an odd number of swaps
        for i, s in enumerate(side):
            sel[i](s)
            M.kv_beam_reorder(tails[i], swap, length, 50, ws[i], s)
    torch.cuda.synchronize()
    for i in range(2):
        sel[i].check(f"stream {i}")
        np.testing.assert_array_equal(t[i].cpu().numpy(), B.beam_reorder(k[i], [[1, 0], [1, 0]], [41] * 4, 2))


def test_beams_of_a_length_above_their_tails(dev):  # noqa: F811
    """A tail that is full: prefix and tail at their bounds, the last row of the cache written."""
    c = _attn_case(41, nh=4, nkv=2, dqk=64, dv=64, plen=[100], tlen=[20, 20], m=3)
    c["kt"], c["vt"] = c["kt"][:, :, :23].copy(), c["vt"][:, :, :23].copy()
    call = Call(c, dev)
    call()
    call.check()


@pytest.mark.parametrize("vocab,k", [(40000, 128), (152577, 64)])
def test_values_of_few_bits(dev, vocab, k):  # noqa: F811
    """Logits as a bfloat16 head leaves them: many equal ones around every border."""
    import torch
    c = _beams(51, 2, 4, vocab, done=True, alpha=0.6)
    c["x"] = torch.from_numpy(c["x"]).bfloat16().float().numpy()
    call = Select(c, k, dev)
    call()
    call.check()


@pytest.mark.parametrize("kw", [
    dict(nh=6, nkv=2, dqk=64, dv=64, plen=[90, 40], tlen=[5, 9, 0, 3], m=5, axes=(12, 10, 10)),
    dict(nh=6, nkv=2, dqk=64, dv=64, plen=[12300], tlen=[5, 9], m=9, axes=(8, 8), rot=32),
    dict(nh=4096, nkv=64, dqk=32, dv=32, plen=[70], tlen=[5], norm=False),
    dict(nh=64, nkv=64, dqk=32, dv=32, plen=[12289], tlen=[5], sinks=True),
    dict(nh=9, nkv=1, dqk=96, dv=160, plen=[33], tlen=[64, 65, 63], m=16, window=70),
])
def test_attention_of_other_layouts(dev, kw):  # noqa: F811
    call = Call(_attn_case(900, **kw), dev)
    call()
    call.check(str(kw))


@pytest.mark.parametrize("plen", [90, 12300])
def test_most_sequences_and_rows(dev, plen):  # noqa: F811
    """1024 sequences of 16 new rows: a few of them against the reference, which takes them alone."""
    c = _attn_case(50, nh=2, nkv=1, dqk=32, dv=32, plen=[plen], tlen=[(5 * i) % 40 - 1 for i in range(1024)], m=16)
    call = Call(c, dev)
    call()
    got, m = call.out.cpu().numpy().reshape(1024, 16, 2, 32), 16
    pick = [0, 1, 7, 511, 512, 777, 1023]
    rows = np.concatenate([np.arange(b * m, b * m + m) for b in pick])
    sub = {**c, "tlen": [c["tlen"][b] for b in pick], "kt": c["kt"][pick], "vt": c["vt"][pick],
           **{n: c[n][rows] for n in ("qp", "kp", "vp")}}
    ref, k, _ = _reference(sub)
    kt = call.kt.cpu().numpy()
    for x, b in enumerate(pick):
        t = c["tlen"][b]
        if t < 0:
            assert (got[b] == 7).all() and np.isnan(kt[b]).all()
        else:
            assert_close(got[b], np.array(ref[x * m:x * m + m]), f"sequence {b}", ATTN_TOL)
            assert_close(kt[b, :, t:t + m], k[x * m:x * m + m].transpose(1, 0, 2), f"keys of {b}", 2e-6)


def test_finished_beams_without_lengths(dev):  # noqa: F811
    """Flags and scores alone, and no new flags wanted."""
    import torch
    import mtp_speculative_draft_gb300 as M
    c = _beams(71, 3, 4, 700, done=True)
    call = Select(c, 5, dev)
    beams = M.beam_set(3, 4, 700, call.score, done=call.done, eos=c["eos"])
    M.beam_select(beams, call.x, 5, call.parent, call.token, call.new_score, ws=call.ws)
    ref = B.beam_select(c["x"], 3, 4, 5, c["score"], done=c["done"], eos=c["eos"])
    torch.cuda.synchronize()
    assert call.parent.tolist() == ref[0].tolist() and call.token.tolist() == ref[1].tolist()
    assert (call.new_length == -9).all() and (call.new_done == -9).all()


def test_lengths_at_the_end_of_their_range(dev):  # noqa: F811
    """2^31 - 1 tokens, and one less: the length stays there."""
    c = _beams(72, 1, 3, 500, alpha=0.5)
    c["length"][:] = 2 ** 31 - 1, 2 ** 31 - 2, 5
    call = Select(c, 3, dev)
    call()
    import torch
    torch.cuda.synchronize()
    want = B.beam_select(c["x"], 1, 3, 3, c["score"], c["length"], alpha=0.5)
    assert call.token.tolist() == want[1].tolist() and call.parent.tolist() == want[0].tolist()
    assert call.new_length[0].tolist() == [min(2 ** 31 - 1, int(c["length"][p]) + 1) for p in call.parent[0].tolist()]


@pytest.mark.parametrize("vocab,k", [(12, 24), (9000, 128)])
def test_logits_at_the_ends_of_their_range(dev, vocab, k):  # noqa: F811
    """Scores below the lowest float: each candidate once, in order, its score -infinity."""
    import torch
    c = _beams(73, 1, 2, vocab)
    if vocab > 100:
        c["x"][0] = -3e38
    c["x"][0, :8] = 3e38, -3e38, 0, 1e30, -1e38, -3.2e38, 2.9e38, 3.1e38
    c["x"][1, 12:] = -np.inf
    call = Select(c, k, dev)
    call()
    torch.cuda.synchronize()
    want = B.beam_select(c["x"], 1, 2, k, c["score"], c["length"])
    assert call.parent.tolist() == want[0].tolist() and call.token.tolist() == want[1].tolist()
    with np.errstate(over="ignore"):
        np.testing.assert_allclose(call.new_score.cpu().numpy(), want[2].astype(np.float32), rtol=2.0 ** -23)
    assert call.new_length.tolist() == want[3].tolist()


@pytest.mark.parametrize("beams,vocab,k,spread", [
    (16, 60000, 32, 1.0), (16, 60001, 17, 40.0), (64, 17000, 64, 3.0), (12, 100000, 128, 1.0), (5, 151936, 33, 1.0)])
@pytest.mark.parametrize("alpha,done", [(0.0, False), (0.7, True)])
def test_selections_of_many_candidates(dev, beams, vocab, k, spread, alpha, done):  # noqa: F811
    """More than a CTA holds at once: chunks by their largest logits first; beams alike and far apart."""
    call = Select(_beams(74, 1, beams, vocab, done, alpha, spread), k, dev)
    call()
    call.check()


def test_most_of_the_chunks_above_the_bound(dev):  # noqa: F811
    """Three good beams of 19 chunks and a bad one: the 64th of the chunks' largest is one of the bad beam's."""
    c = _beams(75, 1, 4, 151936)
    c["score"][3] -= 30
    call = Select(c, 64, dev)
    call()
    call.check()


@pytest.mark.parametrize("k", [1, 16, 33, 128])
def test_equal_logits_in_more_chunks_than_are_listed(dev, k):  # noqa: F811
    """64 equal rows of 19 chunks: the first beam's first tokens."""
    import torch
    c = dict(x=np.zeros((64, 151936), np.float32), seqs=1, beams=64, score=np.full(64, -7, np.float32),
             length=np.full(64, 9, np.int32), done=None, eos=2, alpha=0.5)
    call = Select(c, k, dev)
    call()
    torch.cuda.synchronize()
    assert call.parent[0].tolist() == [0] * k and call.token[0].tolist() == list(range(k))
    np.testing.assert_allclose(call.new_score.cpu().numpy(), -7 - np.log(151936), rtol=2.0 ** -23)


def test_scores_without_bounds_among_many_candidates(dev):  # noqa: F811
    """Logits of +-3e38 in some of many chunks, a row of NaN, one of infinity, one without a token."""
    c = _beams(76, 1, 16, 60000)
    c["x"][0, [0, 9000, 59999]] = 3e38, -3e38, 2.9e38
    c["x"][1] = np.nan
    c["x"][2, 5] = np.inf
    c["x"][3] = -np.inf
    c["x"][4, 8192:] = -np.inf
    call = Select(c, 32, dev)
    call()
    call.check()


def test_lowest_length_of_a_tail_of_several_tiles(dev):  # noqa: F811
    """A length of -2^31 moves nothing, at any row."""
    import torch
    import mtp_speculative_draft_gb300 as M
    k = np.random.default_rng(77).standard_normal((4, 1, 100, 256)).astype(np.float32)
    tk = _t(k, dev)
    tv = tk.clone()
    length = np.array([100, -2 ** 31, 7, -1], np.int32)
    ws = M.kv_beam_reorder(M.kv_tails([tk], [tv], 4), _t(np.array([1, 0, 3, 2], np.int32), dev), _t(length, dev), 100)
    torch.cuda.synchronize()
    assert M.mtp_workspace_status(ws) == 0
    np.testing.assert_array_equal(tk.cpu().numpy(), B.beam_reorder(k, [1, 0, 3, 2], np.maximum(length, 0), 4))
    assert torch.equal(tk, tv)


# Sequences whose keys are many enough that a CTA takes several new rows of them.
def _many_rows(seed, nh, plen, m, window=0, per=160, **kw):
    rng = np.random.default_rng(seed)
    return _attn_case(seed, nh=nh, nkv=1, dqk=64, dv=32, plen=plen, window=window, m=m, sinks=True,
                      tlen=[int(t) for t in rng.integers(-1, 500, per - 3)] + [0, 500, 7], **kw)


@pytest.mark.parametrize("nh,m", [(1, 16), (2, 16), (1, 7), (2, 5)])
@pytest.mark.parametrize("plen,window,kw", [([40], 0, {}), ([300, 123], 200, {}), ([12400], 0, {}), ([12400], 12200, {}),
                                            ([0], 9, dict(per=600)), ([90], 0, dict(axes=(12, 10, 10)))])
def test_several_new_rows_of_few_heads(dev, nh, m, plen, window, kw):  # noqa: F811
    per = kw.get("per", 160) // len(plen) * len(plen)
    call = Call(_many_rows(80 + m, nh, plen, m, window, **{**kw, "per": per}), dev)
    call()
    call.check()


@pytest.mark.parametrize("plen,window,where", [
    (50, 0, "new"), (50, 300, "new"), (50, 300, "tail"), (300, 300, "prompt"), (12500, 0, "new"), (12500, 12400, "new"),
    (12500, 12400, "prompt")])
@pytest.mark.parametrize("nh", [1, 2])
def test_hidden_values_among_several_new_rows(dev, nh, plen, window, where):  # noqa: F811
    """NaN in a later new row's key and value, or below the window of some of the rows: who does not see it gives the
    same result to the bit."""
    m, dv = 8, 32
    c = _many_rows(90, nh, [plen], m, window)
    c["tlen"] = [max(t, 0) for t in c["tlen"]]
    for n in ("kt", "vt"):
        c[n] = np.nan_to_num(c[n])
    clean = Call(c, dev)
    clean()
    clean = clean.out.cpu().numpy().reshape(-1, m, nh, dv)
    bad = []  # positions
    for b, t in enumerate(c["tlen"]):
        at = plen + t + 5 if where == "new" else plen + t + 3 - window if where == "tail" else plen + 250 - window
        if where == "new":
            c["kp"][b * m + 5], c["vp"][b * m + 5] = np.inf, np.nan
        elif where == "tail" and at >= plen:
            c["vt"][b, :, at - plen] = np.nan
        elif where == "prompt":
            c["vpre"][0, :, at] = np.nan
        bad.append(at)
    call = Call(c, dev)
    call()
    got = call.out.cpu().numpy().reshape(-1, m, nh, dv)
    seen = 0
    for b, t in enumerate(c["tlen"]):
        for i in range(m):
            low = max(0, plen + t + i + 1 - window) if window else 0
            if low <= bad[b] <= plen + t + i and (where != "tail" or bad[b] >= plen):
                assert np.isnan(got[b, i]).all(), (b, i)
                seen += 1
            else:
                np.testing.assert_array_equal(got[b, i], clean[b, i])
    assert 0 < seen < len(c["tlen"]) * m and not np.isnan(clean).any()


@pytest.mark.parametrize("kw", [dict(gated=True, rot=20), dict(gated=True, norm=False, pos_base=11), dict(loose=(70, 90))])
@pytest.mark.parametrize("nh,nkv,dim", [(4, 2, 64), (3, 3, 160)])
def test_several_new_rows_gated_and_strided(dev, nh, nkv, dim, kw):  # noqa: F811
    """Gates, some rotated dims, rows with gaps, bounds above the lengths; captured and replayed."""
    import torch
    rng = np.random.default_rng(95)
    c = _attn_case(95, nh=nh, nkv=nkv, dqk=dim, dv=dim, plen=[120, 60], tlen=[int(t) for t in rng.integers(-1, 300, 48)], m=6, **kw)
    call = Call(c, dev, pad=8)
    call()
    call.check()
    first = call.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    call.out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(call.out, first)


@pytest.mark.parametrize("vocab,pad", [(9001, 0), (9002, 0), (20003, 0), (9000, 1), (152577, 0)])
def test_equal_beams_at_every_alignment(dev, vocab, pad):  # noqa: F811
    """Beams of equal rows, scores and lengths whose rows start at different places of a 16-byte word: the lower beam
    first, token by token."""
    c = _beams(78, 2, 4, vocab)
    c["x"][:] = c["x"][0]
    c["score"][:], c["length"][:] = -20.5, 9
    for shift in range(4):
        call = Select(c, 12, dev, shift=shift, pad=pad)
        call()
        call.check(f"shift {shift}")
        assert call.parent.tolist() == [[0, 1, 2, 3] * 3] * 2


@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("depth", [1.0, 4.0, 7.5, 9.0])
@pytest.mark.parametrize("top", [0.0, 3.1])
def test_normaliser_of_tokens_far_below_the_best(dev, depth, spread, top):  # noqa: F811
    """One token at `top` and 7999 about `depth` below it, alike or spread; the beam's score is the normaliser in
    float32, so what is written is their difference.

    In units of 2^-24: a term d below the best is off by d for the rounding of the difference, d for that of the product
    with log2(e), 0.225 d for log2(e) in float32, 4 for the exponential (2^-22), and takes 6 float32 additions; so the
    sum is off by 10 + 2.225 times the mean of d under the softmax.  (8191 tokens of a chunk have a mean of 6.2 at most;
    2^30 tokens 17, of which what lies between the largest logits of chunks takes one rounding more, and a chunk's
    weight 4: 39 units, 2^-18.7.)"""
    import torch
    import mtp_speculative_draft_gb300 as M
    rows, V = 8, 8000
    rng = np.random.default_rng(int(10 * depth))
    x = (top - depth * (1 + 0.01 * np.arange(rows)[:, None]) + rng.uniform(-spread, spread, (rows, V))).astype(np.float32)
    x[:, 77] = top
    d = x[:, 77:78].astype(np.float64) - x
    p = np.exp(-d)
    lse = x[:, 77] + np.log(p.sum(-1))
    score = lse.astype(np.float32)
    i = lambda: torch.empty(rows, 1, dtype=torch.int32, device=dev)  # noqa: E731
    parent, token, out = i(), i(), torch.empty(rows, 1, device=dev)
    M.beam_select(M.beam_set(rows, 1, V, _t(score, dev)), _t(x, dev), 1, parent, token, out)
    assert (token == 77).all()
    want = score + (x[:, 77] - lse)  # the output's own rounding, of a value of 2^-18 or so, is 2^-24 of it
    off = np.abs(out.cpu().numpy()[:, 0] - want)
    bound = (10 + 2.225 * (p * d).sum(-1) / p.sum(-1)) * 2.0 ** -24 + np.abs(want) * 2.0 ** -24
    assert (off <= bound).all(), (off, bound)
