"""Draft-tree calls as a program may make them: streams, devices, layouts, numbers at the ends of their ranges."""

import numpy as np
import pytest

from oracle import tree_oracle as T
from test_gpu_tree import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_largest_counts(dev):  # noqa: F811
    """A path that adds to the largest count of a word, with the prompt's bit and without."""
    import torch
    import mtp_speculative_draft_gb300 as M
    V = 200
    words = np.zeros(V, np.uint32)
    words[[3, 50]], words[[4, 51]], words[[5, 52]] = 0x7FFFFFFF, 0xFFFFFFFF, 0x80000000
    x = np.random.default_rng(1).standard_normal((2, V)).astype(np.float32)
    path = [3, 4, 5, 6, 4]
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.uint32).view(np.int32)).to(dev)  # noqa: E731
    rules = M.logit_rules(V, 1.5, 2.0 ** -20, 0.25, i32(words), path_tokens=i32(path),
                          path_mask=torch.tensor([0b11111, 0], dtype=torch.int64, device=dev))
    out, tok, val = torch.zeros(2, V, device=dev), torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(2, device=dev)
    M.logit_rules_argmax(rules, torch.from_numpy(x).to(dev), tok, val, out)
    ref = T.logit_rules(x, words, 1.5, 2.0 ** -20, 0.25, path_tokens=path, path_mask=[0b11111, 0], dtype=np.float32)
    assert ref[0, 3] < -2000 and ref[0, 4] < -2000  # 2^31 and more
    np.testing.assert_array_equal(out.cpu().numpy(), ref)
    assert tok.tolist() == [t for t, _ in T.greedy(ref)]


def test_workspaces_come_from_the_pool_of_their_stream(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    side = torch.cuda.Stream()
    par = torch.tensor([-1, 0, 0], dtype=torch.int32, device=dev)
    mask, depth = torch.zeros(3, dtype=torch.int64, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    kept = [M.mtp_tree_plan(par, mask, depth, stream=side), M.workspace(100000, stream=side)]
    side.synchronize()
    assert mask.tolist() == [1, 3, 5]
    for ws in kept:
        at = [s["stream"] for s in torch.cuda.memory_snapshot()
              if s["address"] <= ws.data_ptr() < s["address"] + s["total_size"]]
        assert at == [side.cuda_stream]


@pytest.mark.parametrize("rows,d,half", [(1, 64, 32), (37, 64, 32), (5, 128, 30), (300, 96, 16)])
def test_rotation_of_head_major_rows(dev, rows, d, half):  # noqa: F811
    """[heads, rows, head_dim]: queries from such a tensor, keys straight into the rows of a cache, and in place."""
    import torch
    import mtp_speculative_draft_gb300 as M
    from helpers import assert_close
    rng = np.random.default_rng(rows)
    nh, nkv, cap, at = 6, 2, rows + 11, 4
    q, k = (rng.standard_normal((n, rows, d)).astype(np.float32) for n in (nh, nkv))
    w = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    up = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    pos = rng.integers(0, 400, (1, rows)).astype(np.int32)
    table = torch.empty(400 * 2 * half, device=dev)
    M.mtp_rope_table(table, 400, 2 * half, 1e4)
    tq, tk, cache = up(q), up(k), torch.full((nkv, cap, d), float("nan"), device=dev)
    M.rope_axes_rows(M.rope_axes((half,), up(pos), table),
                     [(tq.transpose(0, 1), tq.transpose(0, 1), up(w)),
                      (tk.transpose(0, 1), cache[:, at:at + rows].transpose(0, 1), None)])
    turn = lambda x, w: T.rope_axes(T.head_norm(x.transpose(1, 0, 2), w, 1e-6), pos, (half,), False, 1e4).transpose(1, 0, 2)  # noqa: E731
    assert_close(tq.cpu().numpy(), turn(q, w), "q", 2e-6)  # the roundings of a rotation counted beside its other tests
    assert_close(cache[:, at:at + rows].cpu().numpy(), turn(k, None), "k", 2e-6)
    assert torch.isnan(cache[:, :at]).all() and torch.isnan(cache[:, at + rows:]).all()
    assert (tk == up(k)).all()
    y = torch.zeros(nh, rows, d, device=dev).transpose(0, 1)
    if rows > 1:
        for bad in (tq.transpose(0, 1).as_strided((rows, nh, d), (d // 2, rows * d, 1)),       # rows overlap
                    tq.transpose(0, 1).as_strided((rows, nh, d), (d, (rows - 1) * d, 1))):     # heads overlap
            with pytest.raises(M._lib.MtpError):
                M.rope_axes_rows(M.rope_axes((half,), up(pos), table), [(bad, y, None)])


def test_token_counts_of_the_longest_list(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    n = (1 << 31) - 1
    tokens = torch.full((n,), -1, dtype=torch.int32, device=dev)
    tokens[0], tokens[n - 257], tokens[n - 1] = 3, 4, 3
    counts = torch.zeros(9, dtype=torch.int32, device=dev)
    ws = M.mtp_token_counts(counts, tokens)
    assert counts.tolist() == [0, 0, 0, 2, 1, 0, 0, 0, 0] and M.mtp_workspace_status(ws) == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("eps,scale", [(1e-2, 0.0), (1e-6, 0.3), (0.0, 0.02)])
def test_attention_with_other_scales_and_sections(dev, inter, eps, scale):  # noqa: F811
    """``eps`` and ``scale`` of the geometry, and sections one after another."""
    import test_gpu_tree as G
    from helpers import assert_close
    from mtp_speculative_draft_gb300 import attn_geom, rope_axes
    c = G._attn_case(5, nh=6, nkv=2, dqk=96, dv=64, L=150, n=7, axes=(14, 6, 10), rot=60)
    c["qp"] *= np.float32(0.1)  # eps 0.01 counts
    c["kp"] *= np.float32(0.1)
    call = G.Call(c, dev)
    call.g = attn_geom(6, 2, 96, 64, 60, eps=eps, scale=scale)
    pos, table = call.tree.tensors[2].tensors
    ax = rope_axes((14, 6, 10), pos, table, interleaved=inter)
    call.tree = __import__("mtp_speculative_draft_gb300").draft_tree(*call.tree.tensors[:2], ax)
    call()
    q = T.rope_axes(T.head_norm(c["qp"].reshape(7, 6, 96), c["qn"], eps), c["pos"], (14, 6, 10), inter, 1e4)
    k = T.rope_axes(T.head_norm(c["kp"].reshape(7, 2, 96), c["kn"], eps), c["pos"], (14, 6, 10), inter, 1e4)
    ref = T.tree_attention(q, c["kc"], c["vc"], k, c["vp"].reshape(7, 2, 64), c["mask"], c["depth"],
                           scale=scale if scale else None)
    # logits of three times the usual size at scale 0.3 (1 / sqrt(96) is 0.1)
    assert_close(call.out.cpu().numpy(), ref.reshape(7, -1), "out", 3 * G.ATTN_TOL)


def test_first_call_of_a_process_is_captured(dev):  # noqa: F811
    """Each call's first launch in a process may be under capture."""
    import os
    import subprocess
    import sys
    code = """
import numpy as np, torch
import test_gpu_tree as G
import mtp_speculative_draft_gb300 as M
dev = torch.device("cuda:0")
torch.zeros(1, device=dev)
for kw in (dict(nh=8, nkv=2, dqk=64, dv=64), dict(nh=4, nkv=2, dqk=160, dv=128), dict(nh=4, nkv=2, dqk=64, dv=160)):
    call = G.Call(G._attn_case(3, L=300, n=5, norm=False, rot=0, **kw), dev)
    x, tok, val = torch.randn(2, 9000, device=dev), torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(2, device=dev)
    rules, ws = M.logit_rules(9000), M.workspace(M.logit_rules_argmax_workspace_bytes(2))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        M.logit_rules_argmax(rules, x, tok, val, None, ws)
    g.replay()
    call.check()
    assert (tok == x.argmax(1)).all()
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([here, os.path.dirname(here)])}
    done = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_infinities_in_visible_rows(dev):  # noqa: F811
    """In a new row what the formula gives (a logit of -inf has weight 0), in a cached row that all see NaN."""
    import test_gpu_tree as G
    from helpers import assert_close
    c = G._attn_case(6, nh=4, nkv=2, dqk=64, dv=64, L=100, n=5, rot=0, norm=False, tree="chain")
    c["qp"] = np.abs(c["qp"])
    c["kp"][2, 3] = -np.inf   # KV head 0: nodes 2 to 4 see node 2 with weight 0
    c["vp"][3, 64 + 7] = np.inf  # KV head 1, column 7: infinite for nodes 3 and 4
    call = G.Call(c, dev)
    call()
    got = call.out.cpu().numpy()
    q, k = c["qp"].reshape(5, 4, 64), c["kp"].reshape(5, 2, 64)
    ref = T.tree_attention(q, c["kc"], c["vc"], k, c["vp"].reshape(5, 2, 64), c["mask"], c["depth"]).reshape(5, -1)
    far = np.zeros((5, 4, 64), bool)
    far[3:, 2:, 7] = True
    far = far.reshape(5, -1)
    assert (ref[far] == np.inf).all() and (got[far] == np.inf).all() and np.isfinite(got[~far]).all()
    assert_close(got[~far], ref[~far], "the rest", G.ATTN_TOL)
    c["kc"][1, 50, 9] = -np.inf
    call = G.Call(c, dev)
    call()
    got = call.out.cpu().numpy().reshape(5, 4, 64)
    assert np.isnan(got[:, 2:]).all() and np.isfinite(got[:, :2]).all()
