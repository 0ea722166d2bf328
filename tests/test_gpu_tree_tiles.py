"""Tree attention over long caches: many tiles a split, whose K and V change in size from tile to tile.

The bound of each output is worked out from its own inputs (``exact_and_bound``), from the roundings
of the operands and the sums.  With u = 2^-24 (half a float32 step) and h = 2^-22 (an f16 pair: the
high part is off by 2^-11 of the value at most, the low part by 2^-11 of that):

* a logit: q is scaled (u), q and K are pairs (h each, and 2^-39 of the row's or tile's largest), the
  product of the low parts is left out (h); 3 d / 16 tensor-core steps, each with 17 addends that are
  cut off at 2^-24 of the sum of magnitudes;
* a weight: the logit's error, the subtraction of the reference (u times at most 126 bits that matter),
  ex2 (h);
* the output: the weights' errors times |v| + |o| (numerator and denominator), and relative to the sum
  of magnitudes: pairs of P and V and their left out product (3 h), 3 * 4 tensor-core steps a tile (17 u
  each), a move of the reference a tile (h), the sums over T tiles and over the splits (u each), three
  exponentials of merging (h) and at most 40 further roundings (u); a weight's pair has an absolute error
  of 2^-25, where the largest weight is 2^8 at least, and none above the weight itself: min(p, 2^-33).

Terms of second order are covered by a tenth on top.
"""

import numpy as np
import pytest

from test_gpu_tree import Call, _attn_case, dev  # noqa: F401

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -22


def exact_and_bound(c, splits, tiles):
    """Outputs in 64 bits of a case without norms, rotation, window, sinks and gate, and their bounds."""
    n, nh, nkv, d, dv, L = (c[k] for k in ("n", "nh", "nkv", "dqk", "dv", "L"))
    G, scale = nh // nkv, 1 / np.sqrt(d)
    q = c["qp"].reshape(n, nkv, G, d).transpose(1, 0, 2, 3).reshape(nkv, n * G, d).astype(np.float64)
    kn = c["kp"].reshape(n, nkv, d).transpose(1, 0, 2)
    vn = c["vp"].reshape(n, nkv, dv).transpose(1, 0, 2)
    sees = np.ones((n, L + n), bool)
    sees[:, L:] = [[(int(w) >> j) & 1 for j in range(n)] for w in c["mask"]]
    sees = np.repeat(sees, G, 0)
    out, bound = np.zeros((nkv, n * G, dv)), np.zeros((nkv, n * G, dv))
    for g in range(nkv):
        K = np.concatenate([c["kc"][g], kn[g]]).astype(np.float64)
        V = np.concatenate([c["vc"][g], vn[g]]).astype(np.float64)
        logit = np.where(sees, q[g] @ K.T * scale, -np.inf)
        p = np.exp(logit - logit.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        o = p @ V
        aq, ak, av = np.abs(q[g]), np.abs(K), np.abs(V)
        pairs = 2.0 ** -39 * (aq.max(1, keepdims=True) * ak.sum(1) + ak.max() * aq.sum(1, keepdims=True))
        eps = scale * ((U + 3 * H + 3 * d / 16 * 17 * U) * (aq @ ak.T) + pairs) + 126 * U + H
        assert (p * eps).sum(1).max() < 0.05  # the first order holds
        rel = H * (3 + 3 + tiles) + U * (12 * 17 + tiles + splits + 40)
        mags = p @ av
        bound[g] = 1.1 * ((p * eps) @ av + (p * eps).sum(1, keepdims=True) * np.abs(o) + rel * (mags + np.abs(o)) +
                          np.minimum(p, 2.0 ** -33) @ av + 2.0 ** -38 * av.max())
        out[g] = o
    order = lambda x: x.reshape(nkv, n, G, dv).transpose(1, 0, 2, 3).reshape(n, nh * dv)  # noqa: E731
    return order(out), order(bound)


def tiles_case(seed, pattern, tile, **kw):
    """Rows of tile t of the cache times s(t) (K) and a power of two (V)."""
    c = _attn_case(seed, rot=0, norm=False, **kw)
    t = np.arange(c["L"]) // tile
    s = {"rise": 0.5 * 1.3 ** t, "fall": 0.5 * 1.3 ** (t.max() - t),
         "zigzag": 2.0 ** np.array([0, 4, -3, 2, -6])[t % 5]}[pattern]
    c["kc"] *= np.minimum(s, 32)[None, :, None].astype(np.float32)
    c["vc"] *= (2.0 ** np.array([1, -2, 0, 2, -1])[t % 5])[None, :, None].astype(np.float32)
    return c


def check(call, splits, tiles):
    call()
    got, (out, bound) = call.out.cpu().numpy(), exact_and_bound(call.c, splits, tiles)
    assert np.sqrt(np.mean(bound ** 2)) < 0.05 * np.sqrt(np.mean(out ** 2))  # says something
    assert np.isfinite(got).all()
    worst = np.abs(got - out) / bound
    assert worst.max() <= 1, f"{worst.max():.2f} of the bound at {np.unravel_index(worst.argmax(), worst.shape)}"
    first = call.out.clone()
    for _ in range(3):
        call.out.fill_(7.0)
        call()
        assert (call.out == first).all()


# 64 KV heads have two splits each: ten tiles and more a split
@pytest.mark.parametrize("pattern", ["rise", "fall", "zigzag"])
@pytest.mark.parametrize("group,n,dqk,dv,L", [
    (1, 3, 32, 32, 1300),     # query rows four times in a tile
    (1, 40, 64, 64, 1300),    # twice
    (2, 40, 32, 64, 1300),    # once
    (1, 2, 256, 128, 700),    # tiles of 32 keys, as many operand bytes as fit
    (1, 2, 224, 96, 650),
    (1, 2, 64, 160, 650),     # both warpgroups on one tile
    (1, 2, 256, 256, 650),    # one buffer of V
])
def test_many_tiles(dev, pattern, group, n, dqk, dv, L):  # noqa: F811
    tile = 64 if max(dqk, dv) <= 128 else 32
    c = tiles_case(len(pattern) + L + n, pattern, tile, nh=64 * group, nkv=64, dqk=dqk, dv=dv, L=L, n=n)
    check(Call(c, dev), 2, -(-L // tile))


@pytest.mark.parametrize("n", [2, 64])
@pytest.mark.parametrize("pattern", ["rise", "zigzag"])
def test_32768_keys(dev, n, pattern):  # noqa: F811
    """40 / 8 heads: 27 tiles a split (2 nodes) and 86 (64 nodes)."""
    c = tiles_case(n, pattern, 64 if pattern == "zigzag" else 2048, nh=40, nkv=8, dqk=128, dv=128, L=32768, n=n)
    check(Call(c, dev), 19, 90)


def test_one_workspace_for_every_call_up_to_the_largest(dev):  # noqa: F811
    """Allocated once for 64 nodes and the longest cache, used with fewer of both."""
    from mtp_speculative_draft_gb300 import attn_tree_sink_workspace_bytes, workspace
    kw = dict(nh=40, nkv=8, dqk=128, dv=128)
    calls = [Call(_attn_case(L + n, L=L, n=n, **kw), dev) for L, n in ((1153, 26), (1152, 25), (1152, 16), (300, 51), (65, 1))]
    ws = workspace(attn_tree_sink_workspace_bytes(calls[0].g, 64, 1153))
    for call in calls:
        call.ws = ws
        call()
        call.check()


def test_attention_and_rules_share_a_workspace_in_turn(dev):  # noqa: F811
    """What attention leaves in a workspace is no state of the rules' chunks, and the other way round."""
    import torch
    import mtp_speculative_draft_gb300 as M
    from oracle import tree_oracle as T
    call = Call(_attn_case(31, nh=40, nkv=8, dqk=128, dv=128, L=300, n=16), dev)
    V, x = 9001, np.random.default_rng(4).standard_normal((1024, 9001)).astype(np.float32)
    logits, want = torch.from_numpy(x).to(dev), [t for t, _ in T.greedy(x)]
    call.ws = ws = M.workspace(max(call.ws.numel(), M.logit_rules_argmax_workspace_bytes(1024)))
    tok, val = torch.empty(1024, dtype=torch.int32, device=dev), torch.empty(1024, device=dev)
    for rows in (16, 64, 1024, 1):
        call()
        tok.fill_(-9)
        M.logit_rules_argmax(M.logit_rules(V), logits[:rows], tok, val, None, ws)
        assert tok[:rows].tolist() == want[:rows]
        call.out.fill_(7.0)
        call()
        call.check(f"after rules of {rows} rows")


@pytest.mark.parametrize("dqk,dv", [(64, 64), (64, 160)])
def test_a_row_far_larger_than_its_tile(dev, dqk, dv):  # noqa: F811
    """A key that no query looks at (its logit is far below the others') with a K row 2^20 and a V row 2^24 times
    its tile's: the tile's other values keep an absolute error of 2^-39 of the largest, which the bound counts."""
    c = _attn_case(41, nh=8, nkv=8, dqk=dqk, dv=dv, L=200, n=3, rot=0, norm=False)
    c["qp"] = np.abs(c["qp"])
    c["kc"][:, 70] = -2.0 ** 20
    c["vc"][:, 70] *= np.float32(2.0 ** 24)
    check(Call(c, dev), 19, 4)
